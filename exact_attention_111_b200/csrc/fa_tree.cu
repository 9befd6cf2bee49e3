// fa_tree.cu -- attention of the new tokens of each sequence (one token, a chain, or a tree of
// drafted tokens) over the paged key/value cache, and the merge of units cut between CTAs.
//
// Row (t, g) of key head h is query head h * G + g of new token t.  It sees key position p when p <
// len (the prefix) or when new token p - len is visible to t (mask bit, or p - len <= t):
//     O = sum_p 2^(s_p - m) v_p / sum_p 2^(s_p - m),  s_p = scale * log2(e) * q . k_p,
// in one pass over the keys with a running max m and sum l (online softmax).
//
// This file's kernel is the one for few rows per key head (decoding, small trees), where the cache is
// read once and its bytes are the bound.  One CTA per SM, eight warps that compute and two that load.  A
// chunk is eight steps of 16 or 32 keys, 32 or 64 KB in all, copied by TMA in boxes of whole pages into a ring
// that runs several chunks ahead and on into the next unit; warp w always takes step w.  Each warp
// keeps its own m, l and O; at the end of a segment (the CTA's run of chunks of one unit) the
// eight are merged through shared memory.  (With a ring of its own for each warp, filled by the warp, the
// copies' issue took 700 of a step's 2000 cycles; a ninth warp filling the eight rings was the bottleneck.)
//
// Measured (captured graphs, in bursts): a decoding step of 64 sequences of 1024 to 8191 keys, 32 query and 8 key
// heads of 128, bf16: 177 us, 6.3 TB/s of the cache's bytes (98 % of the copy rate, DRAM 77 % busy by its own
// count); 3 of them are the merge kernel's.  One token over 131072 E4M3 keys, 32 query and 4 key heads of 128: 35 us
// against 21 of bytes; 3 for the merge, and of the 31 of a CTA (58000 cycles) 17 for the fourteen steps of a warp (2280
// cycles each of dependent loads, conversions, products and exponentials, on two warps a scheduler), 7 waiting
// for keys, 6 until the first ones are there.
// One token of 1023 keys, 16 heads of 64: 7.7 us, all latency: 2 until a CTA knows its part, 2 for its
// one chunk, 1 to use and sum it, 1.6 for the merge, the rest between launches.
//
// The products are made transposed, S^T = K Q^T and O^T = V^T P^T (mma.sync m16n8k16): keys and columns
// fill the 16-wide side and rows come in eights, so four or eight query heads of a group cost
// half of what a 16-row tile would, in products, exponentials and registers.
#include <climits>
#include <cmath>

#include "fa.h"
#include "fa_cache.cuh"
#include "sm100.cuh"

namespace fa {

namespace {

constexpr float kLn2f = 0.693147180559945309f;

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// Transposes an 8 x 8 matrix of 16-bit values held as fragments (lane: row lane / 4, columns 2 (lane % 4) ..).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// (volatile: a step's products stay before its stage is released)
template <bool kFp16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kFp16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Whether one of the E4M3 codes or 16-bit floats of w is not finite.
template <bool kFp8, bool kFp16>
__device__ __forceinline__ bool not_finite(uint32_t w) {
  if constexpr (kFp8) {
    return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u;      // 0x7F + 1 carries into bit 7
  } else {
    constexpr uint32_t e = kFp16 ? 0x7C00u : 0x7F80u;
    return (w & e) == e || ((w >> 16) & e) == e;
  }
}

// Asynchronous copy of n <= 16 bytes (the rest of the sixteen zeros), and its arrival on a barrier.
__device__ __forceinline__ void copy16(void* dst, const void* src, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Bytes (i, j) of w, E4M3 codes, as two fp16.
template <int i, int j>
__device__ __forceinline__ uint32_t expand2(uint32_t w) {
  if constexpr (i == 0 && j == 1) return e4m3_to_f16x2(w);
  else if constexpr (i == 2 && j == 3) return e4m3_to_f16x2(w >> 16);
  else return e4m3_to_f16x2(__byte_perm(w, 0, i | (j << 4)));
}

template <int D, bool kFp8>
struct SmallCfg {
  static constexpr int kEsz = kFp8 ? 1 : 2;
  // Keys of a step.  32 where a row is at most 128 bytes: the fixed work of a step (row max, rescale) is
  // then spent on as many bytes as with 16 rows of 256.
  static constexpr int kKeys = D * kEsz <= 128 ? 32 : 16;
  static constexpr int kChunkKeys = 8 * kKeys;           // a chunk: one step of each warp
  static constexpr int kHalf = kChunkKeys * D * kEsz;    // K (or V) of a chunk
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = 3 * 65536 / kStage;
  static constexpr int kRing = kStages * kStage;
  // Merge of the eight warps, eight rows at a time: each warp's O rows (a few floats apart beyond D, so
  // that the fragments' stores spread over the banks), and its rows' statistics.
  static constexpr int kRowF = D + (kFp8 ? 2 : 4);
  static constexpr int kSlotF = 8 * kRowF;
  static constexpr int kStatF = kFp8 ? 24 : 16;           // of a warp: m, l and E4M3's reference of eight rows
  static constexpr int kMerge = kRing, kStats = kMerge + 8 * kSlotF * 4, kBars = kStats + 8 * kStatF * 4;
  // E4M3: the chunks' scale codes, K's then V's
  static constexpr int kCodes = kBars + 2 * kStages * 8 + 16;
  static constexpr int kSmem = kCodes + (kFp8 ? kStages * 2 * kChunkKeys : 0);
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kCodes % 16 == 0, "16-byte copies");
  // 384 threads (the loading warps' warpgroup is completed by two idle ones) x 168 registers at launch,
  // shared out again by setmaxnreg.
  static constexpr int kLaunchRegs = 168, kRegCompute = 216, kRegLoad = 72;
  static_assert(2 * kRegCompute + kRegLoad <= 3 * kLaunchRegs, "register shares");
  static constexpr int kRowB = D * kEsz < 128 ? 64 : 128; // bytes between rows of a 128-byte panel (64-byte rows)
};

// Shared-memory offset of 16-byte chunk c of row r of a step as TMA wrote it; panel: bytes between the
// two 128-byte panels of 256-byte rows.
template <int D, bool kFp8>
__device__ __forceinline__ uint32_t swz(int r, int c, int panel) {
  if constexpr (SmallCfg<D, kFp8>::kRowB == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else if constexpr (D * SmallCfg<D, kFp8>::kEsz == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  else return (c >> 3) * panel + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// kFp16: type of q and o.  A 16-bit cache's products are in that type.  An E4M3 cache's are in fp16, which
// holds every code exactly: K's scale 2^c multiplies the score (32 bits), V's goes into the key's weight,
// 2^(s + c - R) with a reference R of each row's own, which follows the largest s + c that the row has seen: R
// is moved (and O with it) when one is 2^15 above it, to 2^11 under it.  So weights have fp16's full eleven
// bits down to 2^-25 of the row's largest, whatever the scales of other keys: R comes from visible keys
// only.  (One reference for all rows, under the largest scale of a step, was one exponential a weight and
// one maximum a row cheaper, but a scale 2^30 above the others, of a key that a row does not see or gives no
// probability, left that row nothing.)  bf16 queries enter as fp16 with a power of two for each row (row_factor).
template <int D, bool kFp8, bool kFp16, int kNR>
__global__ void __launch_bounds__(384, 1)
    tree_small_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const TreeArgs a) {
  using C = SmallCfg<D, kFp8>;
  constexpr int kG = C::kKeys / 16;                       // 16-key groups
  constexpr bool kMma16 = kFp8 || kFp16;                  // products in fp16
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if ((smem_addr(smem_raw) & 1023u) != 0) {               // the copies' swizzle needs it
    if (threadIdx.x == 0) atomicCAS(a.c.status, 0, kDevBadState);
    return;
  }
  const int warp = warp_id(), lane = lane_id();
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_raw + C::kBars);
  uint64_t* empty = full + C::kStages;
  volatile int* abort_flag = reinterpret_cast<int*>(empty + C::kStages);
  const DevStatus st{a.c.status, a.timeout_ns};

  if (threadIdx.x < C::kStages) {
    mbar_init(&full[threadIdx.x], kFp8 ? 2 + 2 * C::kChunkKeys / 16 : 2);         // both loaders, and their lanes that copy codes
    mbar_init(&empty[threadIdx.x], 8);
  }
  if (threadIdx.x == 0) *abort_flag = 0;
  fence_barrier_init();
  grid_begin();
  if (threadIdx.x == 0) a.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
  const Part part = find_part(a, blockIdx.x == 0 && warp == 0);
  if (part.n == 0) return;
  __syncthreads();

  if (warp >= 8) {
    reg_dec<C::kRegLoad>();
    if (warp > 9) return;
    // ---------------------------------------------------------------- loads: warp 8 K, warp 9 V
    // One chunk at a time: lane i looks up the page of the chunk's 16-key group i (one chunk ahead).  A
    // chunk is loaded when some row of the tile may see its first key.
    const CUtensorMap* map = warp == 8 ? &tm_k : &tm_v;
    const uint8_t* scales = warp == 8 ? a.c.ks : a.c.vs;
    if (lane == 0) prefetch_tmap(map);
    constexpr int kGroups = C::kChunkKeys / 16;
    const int per_box = 1 << (a.c.page_shift - 4);        // groups of a page, and of a copy
    Cursor c = part.at;
    int page = 0;
    auto look_up = [&]() {
      const int pos = c.kt * C::kChunkKeys + 16 * lane;
      if (lane < kGroups && pos < c.s.len + c.s.T)
        page = a.c.table[(long long)c.b * a.c.table_stride + (pos >> a.c.page_shift)];
    };
    look_up();
    int stg = 0, phase = 1, count = 0;                    // chunks loaded
    bool ok = true;
    for (int n = part.n; n > 0 && ok; --n) {
      const int end = c.s.len + c.s.T - c.kt * C::kChunkKeys;     // keys of the chunk from here on do not exist
      int row = (a.c.pages * a.c.Hk) << a.c.page_shift;   // lane's group; past the end: a row behind the
      if (lane < kGroups && 16 * lane < end) {            // tensor reads as zeros
        if ((unsigned)page >= (unsigned)a.c.pages) {
          flag_range(a.c);
          page = 0;                                       // stay inside the cache
        }
        const int pos = c.kt * C::kChunkKeys + 16 * lane;
        row = ((page * a.c.Hk + c.h) << a.c.page_shift) + (pos & ((1 << a.c.page_shift) - 1));
      }
      const bool wanted = c.kt * C::kChunkKeys <= c.last;
      c.kt++;
      if (n > 1) {
        if (c.kt == c.s.KT) next_unit(a, c);
        look_up();
      }
      if (!wanted) continue;
      if (count >= C::kStages) ok = mbar_wait(&empty[stg], phase, abort_flag, st);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      if (lane == 0) mbar_arrive_expect_tx(&full[stg], C::kHalf);
      __syncwarp();
      uint8_t* dst = smem_raw + stg * C::kStage + (warp == 9 ? C::kHalf : 0);
      if (lane < kGroups && lane % per_box == 0) tma_load_3d(dst + lane * 16 * D * C::kEsz, map, &full[stg], 0, row, 0);
      if constexpr (kFp8) {
        if (lane < kGroups) {                             // scale codes, zeros past the end
          const int bytes = min(16, max(0, end - 16 * lane));
          copy16(smem_raw + C::kCodes + (stg * 2 + warp - 8) * C::kChunkKeys + 16 * lane, scales + (bytes > 0 ? row : 0), bytes);
          copy_arrive(&full[stg]);
        }
      }
      ++count;
      if (++stg == C::kStages) {
        stg = 0;
        phase ^= 1;
      }
    }
    // A wait that ran out left copies in flight: let them land before the shared memory goes away.
    if (*abort_flag && lane == 0)
      for (int i = max(0, count - C::kStages); i < count; ++i)
        mbar_wait_drain(&full[i % C::kStages], (i / C::kStages) & 1, st);
    return;
  }

  reg_inc<C::kRegCompute>();
  // this warp's keys in a stage: in a page's copy the panels of 256-byte rows stand one after the other
  const int page_rows = 1 << a.c.page_shift, key0 = warp * C::kKeys;
  const int panel = page_rows * 128;
  const int mine = D * C::kEsz > 128 ? (key0 >> a.c.page_shift) * page_rows * (D * C::kEsz) + (key0 & (page_rows - 1)) * 128
                                     : key0 * D * C::kEsz;
  Cursor rd = part.at;
  int rd_left = part.n;

  // ---------------------------------------------------------------- segments
  const int r0 = lane >> 2, tq = lane & 3;                // fragment row and column quad
  int us = 0, uphase = 0;                                 // stage to use, its parity
  bool ok = true;
  while (rd_left > 0) {
    const SeqView s = rd.s;
    const int h = rd.h;
    const int row0 = (rd.u - h * s.RT) * a.tile_rows;
    const int nrows = min(a.tile_rows, s.T * a.G - row0);
    const bool from_start = rd.kt == 0;
    const int seg_g = part.lo + (part.n - rd_left);       // the segment's first chunk in the line

    // Q fragments: lane / 4 is the row; rows past the unit's last read the last one (never stored).
    // Results and row statistics: rows 2 tq and 2 tq + 1 of each eight.
    uint32_t qf[kNR][D / 16][2];
    int tok[kNR][2];
    float sl2[kNR][2];                                    // score factors
#pragma unroll
    for (int nr = 0; nr < kNR; ++nr) {
      const int r = row0 + min(nr * 8 + r0, nrows - 1);
      const int t = r / a.G, g = r - t * a.G;
      const uint16_t* qp = a.q + (s.cu0 + t) * a.q_tok + (h * a.G + g) * a.q_head;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        if constexpr (kFp8) {
          // the order of the 16 columns of a step is free as long as K's agrees: a lane's
          // four E4M3 columns 4 tq .. 4 tq + 3 stand at places (2tq, 2tq+1, 2tq+8, 2tq+9)
          const uint2 w = *reinterpret_cast<const uint2*>(qp + kk * 16 + 4 * tq);
          qf[nr][kk][0] = w.x;
          qf[nr][kk][1] = w.y;
        } else {
          qf[nr][kk][0] = *reinterpret_cast<const uint32_t*>(qp + kk * 16 + 2 * tq);
          qf[nr][kk][1] = *reinterpret_cast<const uint32_t*>(qp + kk * 16 + 8 + 2 * tq);
        }
      }
      float f = a.scale_log2;
      if constexpr (kFp8 && !kFp16) {
        float amax = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 v = unpack2<false>(qf[nr][kk][i]);
            amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int k = row_factor(amax);
        const float to = scale_value(127 + k);
        f *= scale_value(127 - k);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 v = unpack2<false>(qf[nr][kk][i]);
            qf[nr][kk][i] = pack2<true>(v.x * to, v.y * to);
          }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sl2[nr][e] = kFp8 && !kFp16 ? __shfl_sync(0xffffffffu, f, 4 * (2 * tq + e)) : f;
        tok[nr][e] = __shfl_sync(0xffffffffu, t, 4 * (2 * tq + e));
      }
    }
    // O^T: columns r0 and r0 + 8 (E4M3: 2 r0 and 2 r0 + 1) of each 16, rows 2 tq, 2 tq + 1
    float o[kNR][D / 16][4], m[kNR][2], l[kNR][2], ref[kNR][2];
#pragma unroll
    for (int nr = 0; nr < kNR; ++nr) {
#pragma unroll
      for (int n = 0; n < D / 16; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nr][n][i] = 0.f;
      m[nr][0] = m[nr][1] = -INFINITY;
      l[nr][0] = l[nr][1] = 0.f;
      ref[nr][0] = ref[nr][1] = -INFINITY;                // E4M3: R; otherwise O's reference is m
    }

    // ------------------------------------------------------------ the segment's steps
    // Unit, sequence and head stay; only kt moves until the unit or the part ends.
    const int kt_end = min(s.KT, rd.kt + min(rd_left, s.KT));
    for (int kt = rd.kt; kt < kt_end; ++kt) {
      const int p0 = kt * C::kChunkKeys + key0;
      if (kt * C::kChunkKeys > rd.last) break;            // nor is any chunk after it
      if (ok) ok = mbar_wait(&full[us], uphase, abort_flag, st);
      ok = __all_sync(0xffffffffu, ok);
      if (ok && p0 <= rd.last) {
        const uint8_t* sk = smem_raw + us * C::kStage + mine;
        const uint32_t ak = smem_addr(sk), av = ak + C::kHalf;
        const int end = s.len + s.T - p0;                 // keys of the step from here on do not exist
        const bool masked = p0 + C::kKeys > s.len;
        // ---- S^T = K Q^T, kKeys keys x 8 kNR rows: keys r0 and r0 + 8 of each 16, rows 2 tq, 2 tq + 1
        float sc[kNR][kG][4];
#pragma unroll
        for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
          for (int g = 0; g < kG; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[nr][g][i] = 0.f;
        float kf[kG][2], vf[kG][2];                       // K's scales, V's exponents
        const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lchunk = lane >> 4;
        if constexpr (kFp8) {
#pragma unroll
          for (int c = 0; c < D / 16; c += 2)
#pragma unroll
            for (int g = 0; g < kG; ++g) {
              uint32_t kr[4];
              ldsm4(ak + swz<D, true>(16 * g + lrow, c + lchunk, panel), kr);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t af[4] = {expand2<0, 1>(kr[2 * i]), expand2<0, 1>(kr[2 * i + 1]), expand2<2, 3>(kr[2 * i]),
                                        expand2<2, 3>(kr[2 * i + 1])};
#pragma unroll
                for (int nr = 0; nr < kNR; ++nr) mma16816<true>(sc[nr][g], af, qf[nr][c + i][0], qf[nr][c + i][1]);
              }
            }
          const int ck = smem_raw[C::kCodes + us * 2 * C::kChunkKeys + key0 + lane];
          const int cv = smem_raw[C::kCodes + (us * 2 + 1) * C::kChunkKeys + key0 + lane];
          const float fk = scale_value(ck), fv = (float)(cv - 127);
#pragma unroll
          for (int g = 0; g < kG; ++g)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              kf[g][i] = __shfl_sync(0xffffffffu, fk, 16 * g + 8 * i + r0);
              vf[g][i] = __shfl_sync(0xffffffffu, fv, 16 * g + 8 * i + r0);
            }
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int g = 0; g < kG; ++g) {
              uint32_t kr[4];
              ldsm4(ak + swz<D, false>(16 * g + lrow, 2 * kk + lchunk, panel), kr);
#pragma unroll
              for (int nr = 0; nr < kNR; ++nr) mma16816<kFp16>(sc[nr][g], kr, qf[nr][kk][0], qf[nr][kk][1]);
            }
        }
        // ---- scale, mask, online softmax
        uint32_t pp[kNR][kG][2];                          // P of keys r0 (+ 8), rows 2 tq, 2 tq + 1
        uint32_t see[kNR][2];                             // bit k: key p0 + k is visible to the row
#pragma unroll
        for (int nr = 0; nr < kNR; ++nr) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x[kG][2];
            see[nr][e] = 0xFFFFFFFFu;
#pragma unroll
            for (int g = 0; g < kG; ++g)
#pragma unroll
              for (int i = 0; i < 2; ++i) x[g][i] = sc[nr][g][2 * i + e] * (kFp8 ? sl2[nr][e] * kf[g][i] : sl2[nr][e]);
            if (masked) {
              see[nr][e] = visible32(a, s, tok[nr][e], p0 - s.len);
#pragma unroll
              for (int g = 0; g < kG; ++g)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (!((see[nr][e] >> (16 * g + 8 * i + r0)) & 1u)) x[g][i] = -INFINITY;
            }
            float mx = fmaxf(x[0][0], x[0][1]);
#pragma unroll
            for (int g = 1; g < kG; ++g) mx = max3f(mx, x[g][0], x[g][1]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if (!kFp8 && kMma16) mx -= kFp16Lift;
            const float mn = fmaxf(m[nr][e], mx);
            const float neg = mn == -INFINITY ? 0.f : -mn;
            const float al = ex2(m[nr][e] + neg);         // 0 while m = -inf
            m[nr][e] = mn;
            float sum = 0.f;
#pragma unroll
            for (int g = 0; g < kG; ++g)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float p = ex2(x[g][i] + neg);
                sum += p;
                sc[nr][g][2 * i + e] = p;
              }
            l[nr][e] = l[nr][e] * al + sum;
            float ol = al;                                // O's rescale
            if constexpr (kFp8) {
#pragma unroll
              for (int g = 0; g < kG; ++g)
#pragma unroll
                for (int i = 0; i < 2; ++i) x[g][i] += vf[g][i];
              float my = fmaxf(x[0][0], x[0][1]);
#pragma unroll
              for (int g = 1; g < kG; ++g) my = max3f(my, x[g][0], x[g][1]);
              my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, 4));
              my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, 8));
              my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, 16));
              const float rn = my > ref[nr][e] + 15.f ? my - 11.f : ref[nr][e];
              const float nref = rn == -INFINITY ? 0.f : -rn;
              ol = ex2(ref[nr][e] + nref);
              if (rn == ref[nr][e]) ol = 1.f;             // (-inf as well: O is zero)
              ref[nr][e] = rn;
#pragma unroll
              for (int g = 0; g < kG; ++g)
#pragma unroll
                for (int i = 0; i < 2; ++i) sc[nr][g][2 * i + e] = ex2(x[g][i] + nref);
            }
            if (__any_sync(0xffffffffu, ol != 1.f)) {
#pragma unroll
              for (int n = 0; n < D / 16; ++n) {
                o[nr][n][e] *= ol;
                o[nr][n][2 + e] *= ol;
              }
            }
          }
          // P to 16 bits, one rounding of at most half a step (the row sum keeps 32 bits)
#pragma unroll
          for (int g = 0; g < kG; ++g)
#pragma unroll
            for (int i = 0; i < 2; ++i) pp[nr][g][i] = pack2<kMma16>(sc[nr][g][2 * i], sc[nr][g][2 * i + 1]);
        }
        // ---- O^T += V^T P^T
        // Past the sequence's last key the page holds anything: those rows of V count as zero.  A masked
        // product is 0 * v, which is not 0 where v is not finite: a step of new tokens whose values
        // are not all finite makes its products one by one, visible keys only.
        bool apart = false;
        if (masked) {
          // V's rows that exist, 16 bytes at a time over the warp
          constexpr int kC = D * C::kEsz / 16;            // chunks of a row
          bool bad = false;
#pragma unroll 1
          for (int i = lane; i < min(C::kKeys, end) * kC; i += 32) {
            const uint4 x = *reinterpret_cast<const uint4*>(sk + C::kHalf + swz<D, kFp8>(i / kC, i % kC, panel));
            bad |= not_finite<kFp8, kFp16>(x.x) || not_finite<kFp8, kFp16>(x.y) || not_finite<kFp8, kFp16>(x.z) ||
                   not_finite<kFp8, kFp16>(x.w);
          }
          apart = __any_sync(0xffffffffu, bad);
        }
        if (apart) {
#pragma unroll 1
          for (int key = 0; key < min(C::kKeys, end); ++key) {
            const int src = ((key & 7) << 2) | tq, g = key >> 4, i = (key >> 3) & 1;
            float2 w[kNR];
#pragma unroll
            for (int nr = 0; nr < kNR; ++nr) {
              uint32_t pw = i ? pp[nr][0][1] : pp[nr][0][0];
              if (kG > 1 && g == 1) pw = i ? pp[nr][kG - 1][1] : pp[nr][kG - 1][0];
              w[nr] = unpack2<kMma16>(__shfl_sync(0xffffffffu, pw, src));
            }
#pragma unroll
            for (int n = 0; n < D / 16; ++n)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float x;                                  // V[key][column of accumulators (n, 2 k ..)]
                if constexpr (kFp8) {
                  const int col = 2 * r0 + k;
                  x = unpack2<true>(e4m3_to_f16x2(sk[C::kHalf + swz<D, true>(key, n, panel) + col])).x;
                } else {
                  x = unpack2<kFp16>(*reinterpret_cast<const uint16_t*>(sk + C::kHalf + swz<D, false>(key, 2 * n + k, panel) + 2 * r0)).x;
                }
#pragma unroll
                for (int nr = 0; nr < kNR; ++nr) {
                  if ((see[nr][0] >> key) & 1u) o[nr][n][2 * k] += w[nr].x * x;
                  if ((see[nr][1] >> key) & 1u) o[nr][n][2 * k + 1] += w[nr].y * x;
                }
              }
          }
        } else {
#pragma unroll
          for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
            for (int g = 0; g < kG; ++g)
#pragma unroll
              for (int i = 0; i < 2; ++i) pp[nr][g][i] = transpose8(pp[nr][g][i]);
          auto keep = [&](int g, int i) -> uint32_t {     // keys 16 g + 8 i + 2 tq, + 1
            const int k = end - 16 * g - 2 * tq - 8 * i;
            return (k > 0 ? 0xFFFFu : 0u) | (k > 1 ? 0xFFFF0000u : 0u);
          };
          constexpr int kStep = kFp8 ? 2 : 1;             // 16-column tiles of one load
#pragma unroll
          for (int n = 0; n < D / 16; n += kStep)
#pragma unroll
            for (int g = 0; g < kG; ++g) {
              uint32_t vr[4], af[kStep][4];
              if constexpr (kFp8) {
                ldsm4t(av + swz<D, true>(16 * g + lrow, n + lchunk, panel), vr);
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                  af[i][0] = expand2<0, 2>(vr[2 * i]);
                  af[i][1] = expand2<1, 3>(vr[2 * i]);
                  af[i][2] = expand2<0, 2>(vr[2 * i + 1]);
                  af[i][3] = expand2<1, 3>(vr[2 * i + 1]);
                }
              } else {
                ldsm4t(av + swz<D, false>(16 * g + (lane & 7) + lchunk * 8, 2 * n + ((lane >> 3) & 1), panel), vr);
#pragma unroll
                for (int i = 0; i < 4; ++i) af[0][i] = vr[i];
              }
              if (masked) {
#pragma unroll
                for (int i = 0; i < kStep; ++i)
#pragma unroll
                  for (int k = 0; k < 4; ++k) af[i][k] &= keep(g, k >> 1);
              }
#pragma unroll
              for (int i = 0; i < kStep; ++i)
#pragma unroll
                for (int nr = 0; nr < kNR; ++nr) mma16816<kMma16>(o[nr][n + i], af[i], pp[nr][g][0], pp[nr][g][1]);
            }
        }
      }
      __syncwarp();                                       // the stage has been read
      if (lane == 0) mbar_arrive(&empty[us]);
      us = us + 1 == C::kStages ? 0 : us + 1;
      if (us == 0) uphase ^= 1;
    }
    const bool to_end = kt_end == s.KT;
    rd_left -= kt_end - rd.kt;

    // ------------------------------------------------------------ merge of the eight warps, results
    // Eight rows at a time: every warp leaves its O, m, l (and E) in shared memory, then warp w sums
    // row w.  A whole unit is normalised and stored; a cut one leaves its sums to the merge kernel:
    // slot 0 of this CTA for a segment that began in an earlier CTA, slot 1 for one that only
    // begins here.
    const bool whole = from_start && to_end;
    const int slot = 2 * blockIdx.x + (from_start ? 1 : 0);
    if (threadIdx.x == 0 && from_start && !to_end) {
      a.meta[2 * blockIdx.x] = make_int4(part.line.owner(seg_g + s.KT - 1), nrows, s.cu0, h);
      a.meta[2 * blockIdx.x + 1] = make_int4(row0, 0, 0, 0);
    }
    float* so = reinterpret_cast<float*>(smem_raw + C::kMerge) + warp * C::kSlotF;
    float* stats = reinterpret_cast<float*>(smem_raw + C::kStats);       // [warp][m of 8 rows, l of 8 rows, R of 8 rows]
#pragma unroll
    for (int nr = 0; nr < kNR; ++nr) {
        const int rb = nr * 8;
        if (rb >= nrows) continue;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], 4);
          l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], 8);
          l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], 16);
        }
        if (rb > 0) named_bar_sync(1, 256);                      // the rows before are summed
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* row = so + (2 * tq + e) * C::kRowF;
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            if constexpr (kFp8) {
              *reinterpret_cast<float2*>(row + 16 * n + 2 * r0) = make_float2(o[nr][n][e], o[nr][n][2 + e]);
            } else {
              row[16 * n + r0] = o[nr][n][e];
              row[16 * n + 8 + r0] = o[nr][n][2 + e];
            }
          }
          if (r0 == 0) {
            stats[warp * C::kStatF + 2 * tq + e] = m[nr][e];
            stats[warp * C::kStatF + 8 + 2 * tq + e] = l[nr][e];
            if constexpr (kFp8) stats[warp * C::kStatF + 16 + 2 * tq + e] = ref[nr][e];
          }
        }
        named_bar_sync(1, 256);
        const int r = rb + warp;
        if (r < nrows) {
          constexpr int kV = D / 32;                      // columns of a lane
          float mr = -INFINITY, rr = -INFINITY;
#pragma unroll
          for (int w = 0; w < 8; ++w) {
            mr = fmaxf(mr, stats[w * C::kStatF + warp]);
            if constexpr (kFp8) rr = fmaxf(rr, stats[w * C::kStatF + 16 + warp]);
          }
          const float neg = mr == -INFINITY ? 0.f : -mr, nrr = rr == -INFINITY ? 0.f : -rr;
          float lr = 0.f, x[kV] = {};
#pragma unroll
          for (int w = 0; w < 8; ++w) {
            float f = ex2(stats[w * C::kStatF + warp] + neg);
            lr += f * stats[w * C::kStatF + 8 + warp];
            if constexpr (kFp8) f = ex2(stats[w * C::kStatF + 16 + warp] + nrr);
            const float* src = reinterpret_cast<const float*>(smem_raw + C::kMerge) + w * C::kSlotF + warp * C::kRowF + lane * kV;
#pragma unroll
            for (int i = 0; i < kV; i += 2) {
              const float2 v = *reinterpret_cast<const float2*>(src + i);
              x[i] += f * v.x;
              x[i + 1] += f * v.y;
            }
          }
          if constexpr (kFp8) {                           // O's reference from R to m, 2^(R - m) in two steps: it
            const float f = rr == -INFINITY ? 0.f : ex2(0.5f * (rr + neg));        // may lie outside fp32's normal range
#pragma unroll
            for (int i = 0; i < kV; ++i) x[i] = x[i] * f * f;
          }
          if (whole) {
            const float inv = lr == 0.f ? 0.f : 1.f / lr;
            const int t = (row0 + r) / a.G, g = (row0 + r) - t * a.G;
            const long long tk = s.cu0 + t;
            const int hq = h * a.G + g;
            if (lane == 0) a.lse[tk * a.Hq + hq] = lr == 0.f ? -INFINITY : (mr + log2f(lr)) * kLn2f;
            uint32_t* op = reinterpret_cast<uint32_t*>(a.o + tk * a.o_tok + hq * a.o_head + lane * kV);
#pragma unroll
            for (int i = 0; i < kV; i += 2) op[i / 2] = pack2<kFp16>(x[i] * inv, x[i + 1] * inv);
          } else {
            const long long at = (long long)slot * a.slot_rows + r;
            if (lane == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(mr, lr);
#pragma unroll
            for (int i = 0; i < kV; i += 2)
              *reinterpret_cast<float2*>(a.part_o + at * D + lane * kV + i) = make_float2(x[i], x[i + 1]);
          }
        }
      }
    if (rd_left > 0) named_bar_sync(1, 256);                     // the last rows are summed
    if (rd_left > 0) next_unit(a, rd);
  }
}

// ------------------------------------------------------------------------------------
// Merge of the units cut between CTAs: block (c, y) takes rows of the unit that begins in CTA c and ends
// in a later one.  With parts (m_i, l_i, O_i):
//     O = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i,  m = max_i m_i.
// Few rows (up to 148 parts each): a block has one row, its eight warps share the parts.
// ------------------------------------------------------------------------------------
template <int D, bool kFp16>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeArgs a) {
  constexpr int kV = D / 32;                              // columns per lane
  constexpr int kBatch = 6;                               // parts of a warp whose loads are in flight together
  __shared__ float so[8][D];
  __shared__ float sm[8], sl[8];
  grid_begin();
  const int c = blockIdx.x, lane = lane_id(), warp = warp_id();
  const int4 me = a.meta[2 * c];                          // last CTA, rows, first token, key head
  const int row0 = a.meta[2 * c + 1].x;
  const int r = blockIdx.y;
  if (me.x < 0 || r >= me.y) return;
  const int n = me.x - c + 1;                             // parts: this CTA's and those of c + 1 .. me.x
  // Each warp sums its parts against its own maximum, so that their sums, maxima and values are loaded
  // at once: what counts here is the number of loads that wait for one another.
  float m = -INFINITY, l = 0.f, acc[kV] = {};
  for (int i0 = warp; i0 < n; i0 += 8 * kBatch) {
    float2 ml[kBatch];
    float x[kBatch][kV];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + 8 * j;
      ml[j] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int k = 0; k < kV; ++k) x[j][k] = 0.f;
      if (i < n) {
        const long long at = (2LL * (c + i) + (i == 0 ? 1 : 0)) * a.slot_rows + r;
        ml[j] = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
#pragma unroll
        for (int k = 0; k < kV; k += 2) {
          const float2 v = *reinterpret_cast<const float2*>(a.part_o + at * D + lane * kV + k);
          x[j][k] = v.x;
          x[j][k + 1] = v.y;
        }
      }
    }
    float mn = m;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) mn = fmaxf(mn, ml[j].x);
    const float neg = mn == -INFINITY ? 0.f : -mn;
    const float f = ex2(m + neg);
    m = mn;
    l *= f;
#pragma unroll
    for (int k = 0; k < kV; ++k) acc[k] *= f;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const float w = ex2(ml[j].x + neg);
      l += w * ml[j].y;
#pragma unroll
      for (int k = 0; k < kV; ++k) acc[k] += w * x[j][k];
    }
  }
#pragma unroll
  for (int j = 0; j < kV; ++j) so[warp][lane * kV + j] = acc[j];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  if (warp != 0) return;
  m = -INFINITY;
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, sm[w]);
  const float neg = m == -INFINITY ? 0.f : -m;
  l = 0.f;
#pragma unroll
  for (int j = 0; j < kV; ++j) acc[j] = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const float f = ex2(sm[w] + neg);
    l += f * sl[w];
#pragma unroll
    for (int j = 0; j < kV; ++j) acc[j] += f * so[w][lane * kV + j];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int t = (row0 + r) / a.G, g = (row0 + r) - t * a.G;
  const long long tk = me.z + t;
  const int hq = me.w * a.G + g;
  if (lane == 0) a.lse[tk * a.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2f;
  uint32_t* op = reinterpret_cast<uint32_t*>(a.o + tk * a.o_tok + hq * a.o_head + lane * kV);
#pragma unroll
  for (int j = 0; j < kV; j += 2) op[j / 2] = pack2<kFp16>(acc[j] * inv, acc[j + 1] * inv);
}

// Many rows (the tensor-memory kernel's slots: four columns of all rows, then the next four): a lane has a
// row, a warp eight columns, a block 32 rows and 64 columns.
template <int D, bool kFp16>
__global__ void __launch_bounds__(256) tree_merge_rows_kernel(const TreeArgs a) {
  grid_begin();
  const int c = blockIdx.x, lane = lane_id(), warp = warp_id();
  const int4 me = a.meta[2 * c];                          // last CTA, rows, first token, key head
  const int row0 = a.meta[2 * c + 1].x;
  const int r = (blockIdx.y / (D / 64)) * 32 + lane, col = (blockIdx.y % (D / 64)) * 64 + warp * 8;
  if (me.x < 0 || r >= me.y) return;
  const int n = me.x - c + 1;                             // parts: this CTA's and those of c + 1 .. me.x
  auto slot = [&](int i) { return 2LL * (c + i) + (i == 0 ? 1 : 0); };
  float m = -INFINITY;
  for (int i = 0; i < n; ++i) m = fmaxf(m, a.part_ml[(slot(i) * a.slot_rows + r) * 2]);
  const float neg = m == -INFINITY ? 0.f : -m;
  float l = 0.f, acc[8] = {};
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const long long k = slot(i);
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + (k * a.slot_rows + r) * 2);
    const float w = ex2(ml.x + neg);
    l += w * ml.y;
    const float4* p = reinterpret_cast<const float4*>(a.part_o) + (k * (D / 4) + col / 4) * a.slot_rows + r;
    const float4 x = p[0], y = p[a.slot_rows];
    acc[0] += w * x.x; acc[1] += w * x.y; acc[2] += w * x.z; acc[3] += w * x.w;
    acc[4] += w * y.x; acc[5] += w * y.y; acc[6] += w * y.z; acc[7] += w * y.w;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int t = (row0 + r) / a.G, g = (row0 + r) - t * a.G;
  const long long tk = me.z + t;
  const int hq = me.w * a.G + g;
  if (col == 0) a.lse[tk * a.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2f;
  *reinterpret_cast<uint4*>(a.o + tk * a.o_tok + hq * a.o_head + col) =
      make_uint4(pack2<kFp16>(acc[0] * inv, acc[1] * inv), pack2<kFp16>(acc[2] * inv, acc[3] * inv),
                 pack2<kFp16>(acc[4] * inv, acc[5] * inv), pack2<kFp16>(acc[6] * inv, acc[7] * inv));
}

template <int D, bool kFp8, bool kFp16, int kNR>
cudaError_t launch_small(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, int ctas, cudaStream_t s) {
  auto kern = tree_small_kernel<D, kFp8, kFp16, kNR>;
  constexpr int smem = SmallCfg<D, kFp8>::kSmem;
  static bool done[128];
  const cudaError_t e = prepare_kernel(kern, smem, SmallCfg<D, kFp8>::kLaunchRegs, done);
  if (e != cudaSuccess) return e;
  return launch_after(kern, dim3(ctas), 384, smem, s, tk, tv, a);
}

template <int D, bool kFp8, bool kFp16>
cudaError_t launch_small_nr(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, int ctas, cudaStream_t s) {
  if constexpr (D == 64) {                                 // (most_small)
    if (a.tile_rows == 32) return launch_small<D, kFp8, kFp16, 4>(tk, tv, a, ctas, s);
  }
  return a.tile_rows == 8 ? launch_small<D, kFp8, kFp16, 1>(tk, tv, a, ctas, s) : launch_small<D, kFp8, kFp16, 2>(tk, tv, a, ctas, s);
}

template <int D>
cudaError_t launch_small_d(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, bool fp8, bool fp16,
                           int ctas, cudaStream_t s) {
  if (fp8) return fp16 ? launch_small_nr<D, true, true>(tk, tv, a, ctas, s) : launch_small_nr<D, true, false>(tk, tv, a, ctas, s);
  return fp16 ? launch_small_nr<D, false, true>(tk, tv, a, ctas, s) : launch_small_nr<D, false, false>(tk, tv, a, ctas, s);
}

template <int D, bool kFp16>
cudaError_t launch_merge_d(const TreeArgs& a, int ctas, cudaStream_t s) {
  if (a.tile_rows < kBigRows)
    return launch_after(tree_merge_kernel<D, kFp16>, dim3(ctas, a.slot_rows), 256, 0, s, a);
  return launch_after(tree_merge_rows_kernel<D, kFp16>, dim3(ctas, (a.slot_rows + 31) / 32 * (D / 64)), 256, 0, s, a);
}

struct TreeLayout {
  size_t part_ml, meta, total;
};

// Partial sums of at most two cut units per CTA.
TreeLayout tree_layout(int rows, int d) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  TreeLayout w;
  w.part_ml = up((size_t)kTreeCtas * 2 * rows * d * 4);
  w.meta = w.part_ml + up((size_t)kTreeCtas * 2 * rows * 8);
  w.total = w.meta + up((size_t)kTreeCtas * 2 * sizeof(int4));
  return w;
}

// Most rows of a key head that the few-row kernel takes.  At d = 64 it takes up to 32: 32 sequences of up to 8191 keys,
// 8 key heads, 20 rows 123 us against 141 of the many-row kernel (16 bits) and 135 against 198 (E4M3), 32 rows 107
// against 128 and 117 against 176.  At d = 128 four row blocks spill: 20 rows 305 against 165 (16 bits) and 319 against
// 227 (E4M3), 32 rows 274 against 148 and 272 against 201; up to 16 it is ahead, 123 against 148 and 108 against 211.
int most_small(int d) { return d == 64 ? 32 : 16; }

// Most rows a row tile can have in a call with this many new tokens.
int most_rows(int total, int G) {
  const long long r = ((long long)total * G + 7) / 8 * 8;
  return (int)(r < kBigRows ? r : kBigRows);
}

// Whether the rows of d values of an [n0, n1, d] tensor of these strides lie apart.
bool rows_apart(long long n0, long long s0, long long n1, long long s1, int d) {
  if (n0 <= 1) s0 = LLONG_MAX;
  if (n1 <= 1) s1 = LLONG_MAX;
  const long long lo = s0 < s1 ? s0 : s1, hi = s0 < s1 ? s1 : s0, n = s0 < s1 ? n0 : n1;
  return lo >= d && (hi == LLONG_MAX || (hi - d) / lo >= n - 1);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_fwd_tree_workspace_bytes(int total, int Hq, int Hk, int d) {
  if (total < 0 || Hk < 1 || Hq < Hk || Hq % Hk != 0 || (d != 64 && d != 128)) return 0;
  return tree_layout(most_rows(total > 0 ? total : 1, Hq / Hk), d).total;
}

int fa_fwd_tree(const fa_fwd_tree_args* p) {
  if (p == nullptr) return FA_ERR_INVALID_ARG;
  const fa_fwd_tree_args& x = *p;
  int rc = check_cache(x.cache);
  if (rc != FA_OK) return rc;
  if (x.dtype != FA_BF16 && x.dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  if (x.cache.dtype != FA_E4M3 && x.cache.dtype != x.dtype) return FA_ERR_UNSUPPORTED;
  if (!(x.scale > 0.f) || !std::isfinite(x.scale)) return FA_ERR_INVALID_ARG;
  if (x.total < 0 || x.max_new < 0 || x.Hq < 1 || x.Hq % x.cache.Hk != 0) return FA_ERR_INVALID_ARG;
  if (!x.cu_new || !x.lens || !aligned(x.cu_new, 4) || !aligned(x.lens, 4)) return FA_ERR_INVALID_ARG;
  if (x.tree_mask != nullptr && (x.mask_words < 1 || (long long)x.mask_words * 64 < x.max_new)) return FA_ERR_INVALID_ARG;
  if (!aligned(x.tree_mask, 8)) return FA_ERR_INVALID_ARG;
  // max_new 0 says that there are no new tokens.  With a workspace the kernel looks whether that is so.
  if (x.total == 0 || (x.max_new == 0 && x.workspace == nullptr)) return FA_OK;
  if (!x.q || !x.o || !x.lse || !aligned(x.q, 16) || !aligned(x.o, 16) || !aligned(x.lse, 4)) return FA_ERR_INVALID_ARG;
  for (const long long s : {(long long)x.q_token_stride, (long long)x.q_head_stride, (long long)x.o_token_stride,
                            (long long)x.o_head_stride})
    if (s < 0 || s % 8 != 0) return FA_ERR_INVALID_ARG;
  if (!rows_apart(x.total, x.o_token_stride, x.Hq, x.o_head_stride, x.cache.d)) return FA_ERR_INVALID_ARG;
  const int G = x.Hq / x.cache.Hk;
  if ((long long)x.max_new * G > INT_MAX - 256) return FA_ERR_UNSUPPORTED;
  const TreeLayout w = tree_layout(most_rows(x.total, G), x.cache.d);
  if (!x.workspace || !aligned(x.workspace, 256) || x.workspace_bytes < w.total) return FA_ERR_WORKSPACE;

  const bool fp8 = x.cache.dtype == FA_E4M3, fp16 = x.dtype == FA_FP16;
  TreeArgs a{};
  a.c = view_of(x.cache);
  if (!a.c.status) return FA_ERR_CUDA;
  a.q = static_cast<const uint16_t*>(x.q);
  a.o = static_cast<uint16_t*>(x.o);
  a.lse = x.lse;
  a.cu = x.cu_new;
  a.lens = x.lens;
  a.mask = reinterpret_cast<const unsigned long long*>(x.tree_mask);
  a.words = x.mask_words;
  uint8_t* ws = static_cast<uint8_t*>(x.workspace);
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float*>(ws + w.part_ml);
  a.meta = reinterpret_cast<int4*>(ws + w.meta);
  a.q_tok = x.q_token_stride; a.q_head = x.q_head_stride;
  a.o_tok = x.o_token_stride; a.o_head = x.o_head_stride;
  a.total = x.total;
  a.Hq = x.Hq;
  a.G = G;
  a.max_new = x.max_new;
  a.timeout_ns = 2000000000ull;
  a.scale_log2 = (float)((double)x.scale * 1.4426950408889634);
  const long long unit = (long long)min(x.max_new, x.total) * G;   // most rows of a key head
  const bool big = unit > most_small(x.cache.d);
  a.tile_rows = big ? kBigRows : unit <= 8 ? 8 : unit <= 16 ? 16 : 32;
  a.slot_rows = min(a.tile_rows, most_rows(x.total, G));
  a.chunk_shift = !big && x.cache.d * (fp8 ? 1 : 2) <= 128 ? 8 : 7;   // 32-key steps: SmallCfg

  CUtensorMap tk, tv;
  const long long rows = (long long)x.cache.pages * x.cache.Hk * x.cache.page_size;
  if (!encode_cache(&tk, x.cache.k, rows, x.cache.d, fp8 ? 1 : 2, x.cache.page_size, !big) ||
      !encode_cache(&tv, x.cache.v, rows, x.cache.d, fp8 ? 1 : 2, x.cache.page_size, !big))
    return FA_ERR_CUDA;
  // One CTA per SM, fewer where the longest possible sequences have fewer chunks.
  const long long kt = (((long long)x.cache.max_pages * x.cache.page_size - 1) >> a.chunk_shift) + 1;
  const long long rt = ((long long)x.max_new * G + a.tile_rows - 1) / a.tile_rows;
  long long most = kt * rt;
  most = most > kTreeCtas ? kTreeCtas : most * x.cache.Hk;
  most = most > kTreeCtas ? kTreeCtas : most * x.cache.B;
  const int ctas = (int)(most > kTreeCtas ? kTreeCtas : most < 1 ? 1 : most);       // (max_new 0: one, for the checks)
  const cudaStream_t s = static_cast<cudaStream_t>(x.stream);
  note_launches(0);
  const cudaError_t e = big ? launch_tree_big(tk, tv, a, fp8, fp16, ctas, s)
                        : x.cache.d == 128 ? launch_small_d<128>(tk, tv, a, fp8, fp16, ctas, s)
                                         : launch_small_d<64>(tk, tv, a, fp8, fp16, ctas, s);
  if (e != cudaSuccess) return FA_ERR_CUDA;
  if (kt > 1) {                                            // units of one chunk are never cut
    const cudaError_t em = x.cache.d == 128 ? (fp16 ? launch_merge_d<128, true>(a, ctas, s) : launch_merge_d<128, false>(a, ctas, s))
                                            : (fp16 ? launch_merge_d<64, true>(a, ctas, s) : launch_merge_d<64, false>(a, ctas, s));
    if (em != cudaSuccess) return FA_ERR_CUDA;
  }
  note_launches(kt > 1 ? 2 : 1);
  return FA_OK;
}

}  // extern "C"
