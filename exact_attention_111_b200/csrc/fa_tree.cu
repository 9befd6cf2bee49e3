// fa_tree.cu -- attention of the new tokens of each sequence (one token, a chain, or a tree of
// drafted tokens) over the paged key/value cache, and the merge of units cut between CTAs.
//
// Row (t, g) of key head h is query head h * G + g of new token t.  It sees key position p when p <
// len (the prefix) or when new token p - len is visible to t (mask bit, or p - len <= t):
//     O = sum_p 2^(s_p - m) v_p / sum_p 2^(s_p - m),  s_p = scale * log2(e) * q . k_p,
// in one pass over the keys with a running max m and sum l (online softmax).
//
// This file's kernel is the one for few rows per key head (decoding, small trees), where the cache is
// read once and its bytes are the bound.  One CTA per SM, eight warps.  A chunk of 128 keys is
// eight steps of 16 keys; warp w always takes step w, with a ring of its own that its lane 0 fills by
// TMA several steps ahead, so warps never wait for one another inside a segment and loads cross
// from one unit to the next without a pause.  Each warp keeps its own m, l and O (16 * kMT rows,
// mma.sync m16n8k16 fragments in registers); at the end of a segment (the CTA's run of chunks of one
// unit) the eight are merged through shared memory.
#include <climits>
#include <cmath>

#include "fa.h"
#include "fa_cache.cuh"
#include "sm100.cuh"

namespace fa {

namespace {

constexpr float kLn2f = 0.693147180559945309f;
constexpr int kNoScale = -100000;        // no E yet: below every scale code

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool kFp16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kFp16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
  // Keys of a step.  32 where a row is at most 128 bytes: the fixed work of a step (its copies, row
  // max and rescale) is then spent on 8 KB as with 16 rows of 256 bytes.
  static constexpr int kKeys = D * kEsz <= 128 ? 32 : 16;
  static constexpr int kChunkKeys = 8 * kKeys;           // a chunk: one step of each warp
  static constexpr int kBoxes = kKeys / 16;              // copies of 16 rows (a page holds at least 16)
  static constexpr int kBox = 16 * D * kEsz;
  static constexpr int kHalf = kBoxes * kBox;            // K (or V) of a step
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = 24576 / kStage;
  static constexpr int kRing = 8 * kStages * kStage;     // all warps
  static constexpr int kSlot = 16 * (D / 2) * 4 + 144;   // half of one warp's O, its m, l and E, of 16 rows
  static constexpr int kScales = kFp8 ? 8 * kStages * 2 * kKeys : 0;
  static constexpr int kSmem = kRing + 4 * kSlot + kScales;
  // bytes between 16-byte chunks' rows: 128-byte panels (64-byte rows for E4M3 at d = 64)
  static constexpr int kRowB = D * kEsz < 128 ? 64 : 128;
};

// Shared-memory offset of 16-byte chunk c of row r of K or V of a step as TMA wrote it.
template <int D, bool kFp8>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  const uint32_t box = (r >> 4) * SmallCfg<D, kFp8>::kBox;
  if constexpr (SmallCfg<D, kFp8>::kRowB == 64) return box + (r & 15) * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else return box + (c >> 3) * 2048 + (r & 15) * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// kFp16: type of q and o.  A 16-bit cache's products are in that type.  An E4M3 cache's are in fp16, which
// holds every code exactly: K's scale multiplies the score (32 bits), V's the probability before it
// is rounded, p * 2^(e - E) with E a warp's own reference: 2^8 under the scales of its first keys,
// moved (and O with it) when a scale is 2^15 above it.  So p * 2^(e - E) has fp16's full eleven
// bits down to 2^-22 for keys of the usual scale, three more than bf16.  bf16 queries enter as fp16 with a
// power of two for each row (row_factor).
template <int D, bool kFp8, bool kFp16, int kMT>
__global__ void __launch_bounds__(256, 1)
    tree_small_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const TreeArgs a) {
  using C = SmallCfg<D, kFp8>;
  constexpr int kNT = D / 8;                              // 8-column tiles of O
  constexpr int kST = C::kKeys / 8;                       // 8-key tiles of S
  constexpr int kG = C::kKeys / 16;                       // 16-key groups
  constexpr bool kMma16 = kFp8 || kFp16;                  // products in fp16
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint64_t full[8][C::kStages];
  __shared__ int abort_flag;
  if ((smem_addr(smem_raw) & 1023u) != 0) {               // the copies' swizzle needs it
    if (threadIdx.x == 0) atomicCAS(a.c.status, 0, kDevBadState);
    return;
  }
  const int warp = warp_id(), lane = lane_id();
  uint8_t* ring = smem_raw + warp * C::kStages * C::kStage;
  uint8_t* slots = smem_raw + C::kRing;
  uint8_t* scales = slots + 4 * C::kSlot + warp * C::kStages * 2 * C::kKeys;
  const DevStatus st{a.c.status, a.timeout_ns};

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (lane == 0)
    for (int i = 0; i < C::kStages; ++i) mbar_init(&full[warp][i], 1);
  if (threadIdx.x == 0) {
    abort_flag = 0;
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  fence_barrier_init();

  const long long total = total_chunks(a, blockIdx.x == 0 && warp == 0);
  const Part part = part_of(total, blockIdx.x, gridDim.x);
  if (threadIdx.x == 0) a.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
  if (part.n == 0) return;
  Cursor rd = locate(a, part.lo), ld = rd;
  int rd_left = part.n, ld_left = part.n;
  __syncthreads();

  // ---------------------------------------------------------------- loads
  // A step is loaded when its first key exists and some row of the tile may see it.  `ld` stands at
  // the next step to load, whose page ids (lane i: box i) are on their way since the last.
  auto wanted = [&](const Cursor& c) { return c.kt * C::kChunkKeys + warp * C::kKeys <= c.last; };
  int page = 0;
  auto advance = [&](Cursor& c, int& left) {
    --left;
    if (++c.kt < c.s.KT) return;
    if (left > 0) next_unit(a, c);
  };
  auto look_up = [&]() {
    while (ld_left > 0 && !wanted(ld)) advance(ld, ld_left);
    if (ld_left > 0 && lane < C::kBoxes) {
      const int pos = ld.kt * C::kChunkKeys + warp * C::kKeys + 16 * lane;
      if (pos < ld.s.len + ld.s.T) page = a.c.table[(long long)ld.b * a.c.table_stride + (pos >> a.c.page_shift)];
    }
  };
  int fs = 0;                                             // stage to fill
  auto fill = [&]() {                                     // start the next wanted step's copies, if any
    if (ld_left <= 0) return;
    const int p0 = ld.kt * C::kChunkKeys + warp * C::kKeys, end = ld.s.len + ld.s.T;
    uint64_t* bar = &full[warp][fs];
    if (lane == 0) {
      const int boxes = min(C::kBoxes, (end - p0 + 15) >> 4);     // that hold keys: scales come with them
      mbar_arrive_expect_tx(bar, C::kStage + (kFp8 ? boxes * 32 : 0));
    }
    __syncwarp();
    if (lane < C::kBoxes) {
      const int pos = p0 + 16 * lane;
      int row;
      if (pos >= end) {                                   // past the end: a row behind the tensor reads as zeros
        row = (a.c.pages * a.c.Hk) << a.c.page_shift;
      } else {
        if ((unsigned)page >= (unsigned)a.c.pages) {
          flag_range(a.c);
          page = 0;                                       // stay inside the cache
        }
        row = ((page * a.c.Hk + ld.h) << a.c.page_shift) + (pos & ((1 << a.c.page_shift) - 1));
      }
      uint8_t* dst = ring + fs * C::kStage + lane * C::kBox;
      tma_load_3d(dst, &tm_k, bar, 0, row, 0);
      tma_load_3d(dst + C::kHalf, &tm_v, bar, 0, row, 0);
      if constexpr (kFp8) {
        if (pos < end) {
          bulk_load(scales + fs * 2 * C::kKeys + 16 * lane, a.c.ks + row, 16, bar);
          bulk_load(scales + (fs * 2 + 1) * C::kKeys + 16 * lane, a.c.vs + row, 16, bar);
        }
      }
    }
    fs = fs + 1 == C::kStages ? 0 : fs + 1;
    advance(ld, ld_left);
    look_up();
  };
  look_up();
  int issued = 0;
  for (int i = 0; i < C::kStages && ld_left > 0; ++i, ++issued) fill();

  // ---------------------------------------------------------------- segments
  const int r0 = lane >> 2, tq = lane & 3;                // fragment row and column quad
  int us = 0, uphase = 0, used = 0;                       // stage to use, its parity
  bool ok = true;
  while (rd_left > 0) {
    const SeqView s = rd.s;
    const int h = rd.h;
    const int row0 = (rd.u - h * s.RT) * a.tile_rows;
    const int nrows = (int)min((long long)a.tile_rows, (long long)s.T * a.G - row0);
    const bool from_start = rd.kt == 0;
    const long long seg_g = part.lo + (part.n - rd_left);  // the segment's first chunk in the line

    // Q fragments; rows past the unit's last read the last one (never stored)
    uint32_t qf[kMT][D / 16][4];
    int tok[kMT][2];
    float sl2[kMT][2];                                    // score factors of the lane's rows
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int r = row0 + min(mt * 16 + hf * 8 + r0, nrows - 1);
        const int t = r / a.G, g = r - t * a.G;
        tok[mt][hf] = t;
        const uint16_t* qp = a.q + (s.cu0 + t) * a.q_tok + (h * a.G + g) * a.q_head;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          if constexpr (kFp8) {
            // the order of the 16 columns of a step is free as long as K's agrees: a lane's
            // four E4M3 columns 4 tq .. 4 tq + 3 stand at places (2tq, 2tq+1, 2tq+8, 2tq+9)
            const uint2 w = *reinterpret_cast<const uint2*>(qp + kk * 16 + 4 * tq);
            qf[mt][kk][hf] = w.x;
            qf[mt][kk][hf + 2] = w.y;
          } else {
            qf[mt][kk][hf] = *reinterpret_cast<const uint32_t*>(qp + kk * 16 + 2 * tq);
            qf[mt][kk][hf + 2] = *reinterpret_cast<const uint32_t*>(qp + kk * 16 + 8 + 2 * tq);
          }
        }
        sl2[mt][hf] = a.scale_log2;
        if constexpr (kFp8 && !kFp16) {
          float amax = 0.f;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              const float2 f = unpack2<false>(qf[mt][kk][hf + i]);
              amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          const int k = row_factor(amax);
          const float f = scale_value(127 + k);
          sl2[mt][hf] *= scale_value(127 - k);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              const float2 v = unpack2<false>(qf[mt][kk][hf + i]);
              qf[mt][kk][hf + i] = pack2<true>(v.x * f, v.y * f);
            }
        }
      }
    float o[kMT][kNT][4], m[kMT][2], l[kMT][2];
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[mt][n][i] = 0.f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
    }
    int eref = kNoScale;                                  // E4M3: E (as a scale code) of what O holds

    // ------------------------------------------------------------ the segment's steps
    // Unit, sequence and head stay; only kt moves until the unit or the part ends.
    const int kt_end = (int)min((long long)s.KT, (long long)rd.kt + rd_left);
    for (int kt = rd.kt; kt < kt_end; ++kt) {
      const int p0 = kt * C::kChunkKeys + warp * C::kKeys;
      if (p0 > rd.last) continue;
      if (ok) ok = mbar_wait(&full[warp][us], uphase, &abort_flag, st);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        const uint8_t* sk = ring + us * C::kStage;
        const uint32_t ak = smem_addr(sk), av = ak + C::kHalf;
        const int end = s.len + s.T - p0;                 // keys of the step from here on do not exist
        const bool masked = p0 + C::kKeys > s.len;
        // ---- S = Q K^T, 16 * kMT rows x kKeys keys
        float sc[kMT][kST][4];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int j = 0; j < kST; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[mt][j][i] = 0.f;
        float kf[kST][2], vf[kST][2];
        if constexpr (kFp8) {
          const uint8_t* sp = scales + us * 2 * C::kKeys;
#pragma unroll
          for (int c = 0; c < D / 16; c += 2)
#pragma unroll
            for (int g = 0; g < kG; ++g) {
              uint32_t kr[4];
              ldsm4(ak + swz<D, true>(16 * g + (lane & 7) + ((lane >> 3) & 1) * 8, c + (lane >> 4)), kr);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t a0 = expand2<0, 1>(kr[j]), a1 = expand2<2, 3>(kr[j]);
                const uint32_t b0 = expand2<0, 1>(kr[2 + j]), b1 = expand2<2, 3>(kr[2 + j]);
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) {
                  mma16816<true>(sc[mt][2 * g + j], qf[mt][c], a0, a1);
                  mma16816<true>(sc[mt][2 * g + j], qf[mt][c + 1], b0, b1);
                }
              }
            }
          // the largest of V's scales among the keys that exist
          const uint32_t top = __reduce_max_sync(0xffffffffu, lane < min(C::kKeys, end) ? sp[C::kKeys + (lane & (C::kKeys - 1))] : 0u);
          if ((int)top > eref + 15) {
            const int e = (int)top - 8;
            if (eref != kNoScale) {                       // rare: a scale far above the ones before
              const float f = exp2f((float)(eref - e));
#pragma unroll
              for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                  for (int i = 0; i < 4; ++i) o[mt][n][i] *= f;
            }
            eref = e;
          }
#pragma unroll
          for (int j = 0; j < kST; ++j) {
            const int wk = *reinterpret_cast<const uint16_t*>(sp + 8 * j + 2 * tq);
            const int wv = *reinterpret_cast<const uint16_t*>(sp + C::kKeys + 8 * j + 2 * tq);
            kf[j][0] = scale_value(wk & 0xFF);
            kf[j][1] = scale_value(wk >> 8);
            vf[j][0] = scale_value(max((wv & 0xFF) + 127 - eref, 0));
            vf[j][1] = scale_value(max((wv >> 8) + 127 - eref, 0));
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int g = 0; g < kG; ++g) {
              uint32_t kr[4];
              ldsm4(ak + swz<D, false>(16 * g + (lane & 7) + (lane >> 4) * 8, 2 * kk + ((lane >> 3) & 1)), kr);
#pragma unroll
              for (int mt = 0; mt < kMT; ++mt) {
                mma16816<kFp16>(sc[mt][2 * g], qf[mt][kk], kr[0], kr[1]);
                mma16816<kFp16>(sc[mt][2 * g + 1], qf[mt][kk], kr[2], kr[3]);
              }
            }
        }
        // ---- scale, mask, online softmax
        uint32_t pf[kMT][kG][4];
        unsigned see[kMT][2];                             // bit 2j + i: key 8j + 2 tq + i is visible
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float x[kST][2];
            see[mt][hf] = 0xFFu;
#pragma unroll
            for (int j = 0; j < kST; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i) x[j][i] = sc[mt][j][2 * hf + i] * (kFp8 ? sl2[mt][hf] * kf[j][i] : sl2[mt][hf]);
            if (masked) {
              const int t = tok[mt][hf];
#pragma unroll
              for (int j = 0; j < kST; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int n = p0 + 8 * j + 2 * tq + i - s.len;     // new token of this key
                  bool vis = n < 0;
                  if (n >= 0 && n < s.T) {
                    if (a.mask == nullptr) vis = n <= t;
                    else vis = (n >> 6) < a.words &&
                               ((a.mask[(long long)(s.cu0 + t) * a.words + (n >> 6)] >> (n & 63)) & 1);
                  }
                  if (!vis) {
                    x[j][i] = -INFINITY;
                    see[mt][hf] &= ~(1u << (2 * j + i));
                  }
                }
            }
            float mx = fmaxf(x[0][0], x[0][1]);
#pragma unroll
            for (int j = 1; j < kST; ++j) mx = max3f(mx, x[j][0], x[j][1]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[mt][hf], mx);
            const float neg = mn == -INFINITY ? 0.f : -mn;
            const float al = ex2(m[mt][hf] + neg);        // 0 while m = -inf
            m[mt][hf] = mn;
            float sum = 0.f;
            float p[kST][2];
#pragma unroll
            for (int j = 0; j < kST; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                p[j][i] = ex2(x[j][i] + neg);
                sum += p[j][i];
              }
            l[mt][hf] = l[mt][hf] * al + sum;
            if (__any_sync(0xffffffffu, al != 1.f)) {
#pragma unroll
              for (int n = 0; n < kNT; ++n) {
                o[mt][n][2 * hf] *= al;
                o[mt][n][2 * hf + 1] *= al;
              }
            }
            // P to 16 bits, one rounding of at most half a step (the row sum keeps 32 bits); a
            // masked key's scale may be anything, so its zero is not multiplied
#pragma unroll
            for (int j = 0; j < kST; ++j) {
              if constexpr (kFp8) {
#pragma unroll
                for (int i = 0; i < 2; ++i) p[j][i] = masked && !((see[mt][hf] >> (2 * j + i)) & 1) ? 0.f : p[j][i] * vf[j][i];
              }
              pf[mt][j >> 1][hf + 2 * (j & 1)] = pack2<kMma16>(p[j][0], p[j][1]);
            }
          }
        }
        // ---- O += P V
        // V of a 16-key group, columns 32 c .. 32 c + 31 (E4M3) or 16 c .. 16 c + 15: kVT tiles of 8
        constexpr int kVT = kFp8 ? 4 : 2;
        auto vfrag = [&](int g, int c, uint32_t (&b)[kVT][2]) {
          uint32_t vr[4];
          ldsm4t(av + swz<D, kFp8>(16 * g + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * c + (lane >> 4)), vr);
#pragma unroll
          for (int i = 0; i < 4; ++i) {                   // keys 8 (i % 2) .., 16-byte chunk i / 2
            if constexpr (kFp8) {
              b[2 * (i >> 1)][i & 1] = expand2<0, 2>(vr[i]);
              b[2 * (i >> 1) + 1][i & 1] = expand2<1, 3>(vr[i]);
            } else {
              b[i >> 1][i & 1] = vr[i];
            }
          }
        };
        // Past the sequence's last key the page holds anything: those rows of V count as zero.
        auto keep = [&](int g, int i) -> uint32_t {       // of the keys in half i of group g's fragments
          const int k = end - 16 * g - 2 * tq - 8 * i;
          return (k > 0 ? 0xFFFFu : 0u) | (k > 1 ? 0xFFFF0000u : 0u);
        };
        // A masked product is 0 * v, which is not 0 where v is not finite: a step of new tokens
        // whose values are not all finite makes its products one by one, visible keys only.
        bool apart = false;
        if (masked) {
          bool bad = false;
#pragma unroll 1
          for (int c = 0; c < kNT / kVT; ++c)
#pragma unroll
            for (int g = 0; g < kG; ++g) {
              uint32_t b[kVT][2];
              vfrag(g, c, b);
#pragma unroll
              for (int i = 0; i < 2 * kVT; ++i) {
                const uint32_t w = b[i >> 1][i & 1] & keep(g, i & 1);
                const uint32_t e = kMma16 ? 0x7C00u : 0x7F80u;
                bad |= (w & e) == e || ((w >> 16) & e) == e;
              }
            }
          apart = __any_sync(0xffffffffu, bad);
        }
        if (apart) {
#pragma unroll 1
          for (int key = 0; key < min(C::kKeys, end); ++key) {
            const int src = (lane & ~3) | ((key & 7) >> 1), j = key >> 3, i = key & 1;
            float w[kMT][2];
            bool v[kMT][2];
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                uint32_t pw = pf[mt][0][hf];              // tile j's pair of this lane's row
#pragma unroll
                for (int k = 1; k < kST; ++k)
                  if (j == k) pw = pf[mt][k >> 1][hf + 2 * (k & 1)];
                const float2 f = unpack2<kMma16>(__shfl_sync(0xffffffffu, pw, src));
                w[mt][hf] = i ? f.y : f.x;
                v[mt][hf] = (__shfl_sync(0xffffffffu, see[mt][hf], src) >> (2 * j + i)) & 1;
              }
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float x;                                  // V[key][column of accumulator (n, e)]
                if constexpr (kFp8) {
                  const int col = 16 * (n >> 1) + 4 * tq + 2 * e + (n & 1);
                  x = unpack2<true>(e4m3_to_f16x2(sk[C::kHalf + swz<D, true>(key, col >> 4) + (col & 15)])).x;
                } else {
                  const int col = 8 * n + 2 * tq + e;
                  x = unpack2<kFp16>(*reinterpret_cast<const uint16_t*>(sk + C::kHalf + swz<D, false>(key, col >> 3) +
                                                                        2 * (col & 7))).x;
                }
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                  for (int hf = 0; hf < 2; ++hf)
                    if (v[mt][hf]) o[mt][n][2 * hf + e] += w[mt][hf] * x;
              }
          }
        } else {
#pragma unroll
          for (int c = 0; c < kNT / kVT; ++c)
#pragma unroll
            for (int g = 0; g < kG; ++g) {
              uint32_t b[kVT][2];
              vfrag(g, c, b);
              if (masked) {
#pragma unroll
                for (int i = 0; i < 2 * kVT; ++i) b[i >> 1][i & 1] &= keep(g, i & 1);
              }
#pragma unroll
              for (int i = 0; i < kVT; ++i)
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) mma16816<kMma16>(o[mt][kVT * c + i], pf[mt][g], b[i][0], b[i][1]);
            }
        }
      }
      us = us + 1 == C::kStages ? 0 : us + 1;
      if (us == 0) uphase ^= 1;
      ++used;
      __syncwarp();                                       // the stage has been read: refill it
      if (ok && ld_left > 0) {
        fill();
        ++issued;
      }
    }
    const bool to_end = kt_end == s.KT;
    rd_left -= kt_end - rd.kt;

    // ------------------------------------------------------------ merge of the eight warps
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        l[mt][hf] += __shfl_xor_sync(0xffffffffu, l[mt][hf], 1);
        l[mt][hf] += __shfl_xor_sync(0xffffffffu, l[mt][hf], 2);
      }
      int em = eref;                                      // E of this row block's O
      for (int half = 4; half > 0; half >>= 1) {
        float fa[2], fb[2];
#pragma unroll
        for (int part2 = 0; part2 < 2; ++part2) {         // half of the columns at a time
          constexpr int kH = kNT / 2;
          __syncthreads();
          if (warp >= half && warp < 2 * half) {
            uint8_t* sl = slots + (warp - half) * C::kSlot;
            float4* so = reinterpret_cast<float4*>(sl);
#pragma unroll
            for (int n = 0; n < kH; ++n) {
              const float (&x)[4] = o[mt][part2 * kH + n];
              so[n * 32 + lane] = make_float4(x[0], x[1], x[2], x[3]);
            }
            float* sm = reinterpret_cast<float*>(sl + 16 * (D / 2) * 4);
            if (part2 == 0 && tq == 0) {
              sm[r0] = m[mt][0];
              sm[r0 + 8] = m[mt][1];
              sm[16 + r0] = l[mt][0];
              sm[24 + r0] = l[mt][1];
            }
            if (kFp8 && part2 == 0 && lane == 0) reinterpret_cast<int*>(sm)[32] = em;
          }
          __syncthreads();
          if (warp < half) {
            const uint8_t* sl = slots + warp * C::kSlot;
            const float4* so = reinterpret_cast<const float4*>(sl);
            if (part2 == 0) {
              const float* sm = reinterpret_cast<const float*>(sl + 16 * (D / 2) * 4);
              float ga = 1.f, gb = 1.f;                   // factors of O beside the maxima's
              if constexpr (kFp8) {
                const int eb = reinterpret_cast<const int*>(sm)[32], en = max(em, eb);
                ga = exp2f((float)(em - en));
                gb = exp2f((float)(eb - en));
                em = en;
              }
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                const float mb = sm[r0 + 8 * hf], lb = sm[16 + r0 + 8 * hf];
                const float mn = fmaxf(m[mt][hf], mb);
                const float neg = mn == -INFINITY ? 0.f : -mn;
                fa[hf] = ex2(m[mt][hf] + neg);
                fb[hf] = ex2(mb + neg);
                m[mt][hf] = mn;
                l[mt][hf] = l[mt][hf] * fa[hf] + lb * fb[hf];
                fa[hf] *= ga;
                fb[hf] *= gb;
              }
            }
#pragma unroll
            for (int n = 0; n < kH; ++n) {
              const float4 w = so[n * 32 + lane];
              float (&x)[4] = o[mt][part2 * kH + n];
              x[0] = x[0] * fa[0] + w.x * fb[0];
              x[1] = x[1] * fa[0] + w.y * fb[0];
              x[2] = x[2] * fa[1] + w.z * fb[1];
              x[3] = x[3] * fa[1] + w.w * fb[1];
            }
          }
        }
      }
      if (mt == kMT - 1) eref = em;
    }

    // ------------------------------------------------------------ results
    // A whole unit is normalised and stored; a cut one leaves its sums to the merge: slot 0 of this
    // CTA for a segment that began in an earlier CTA, slot 1 for one that only begins here.
    if (warp == 0) {
      const bool whole = from_start && to_end;
      const int slot = 2 * blockIdx.x + (from_start ? 1 : 0);
      if (lane == 0 && from_start && !to_end) {
        a.meta[2 * blockIdx.x] = make_int4(owner_cta(total, seg_g + s.KT - 1, gridDim.x), nrows, s.cu0, h);
        a.meta[2 * blockIdx.x + 1] = make_int4(row0, 0, 0, 0);
      }
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int r = mt * 16 + hf * 8 + r0;
          if (r >= nrows) continue;
          const float lv = l[mt][hf];
          // what O is a multiple of: 2^(E - 127)
          const float vref = kFp8 && eref != kNoScale ? exp2f((float)(eref - 127)) : 1.f;
          if (whole) {
            const float inv = lv == 0.f ? 0.f : vref / lv;
            const int t = (row0 + r) / a.G, g = (row0 + r) - t * a.G;
            const long long tk = s.cu0 + t;
            const int hq = h * a.G + g;
            if (tq == 0) a.lse[tk * a.Hq + hq] = lv == 0.f ? -INFINITY : (m[mt][hf] + log2f(lv)) * kLn2f;
            uint16_t* op = a.o + tk * a.o_tok + hq * a.o_head;
            if constexpr (kFp8) {
#pragma unroll
              for (int c = 0; c < D / 16; ++c)
                *reinterpret_cast<uint2*>(op + 16 * c + 4 * tq) =
                    make_uint2(pack2<kFp16>(o[mt][2 * c][2 * hf] * inv, o[mt][2 * c + 1][2 * hf] * inv),
                               pack2<kFp16>(o[mt][2 * c][2 * hf + 1] * inv, o[mt][2 * c + 1][2 * hf + 1] * inv));
            } else {
#pragma unroll
              for (int n = 0; n < kNT; ++n)
                *reinterpret_cast<uint32_t*>(op + 8 * n + 2 * tq) =
                    pack2<kFp16>(o[mt][n][2 * hf] * inv, o[mt][n][2 * hf + 1] * inv);
            }
          } else {
            float* pp = a.part_o + ((long long)slot * a.slot_rows + r) * D;
            if (tq == 0) {
              float* ml = a.part_ml + ((long long)slot * a.slot_rows + r) * 2;
              ml[0] = m[mt][hf];
              ml[1] = lv;
            }
            if constexpr (kFp8) {
#pragma unroll
              for (int c = 0; c < D / 16; ++c)
                *reinterpret_cast<float4*>(pp + 16 * c + 4 * tq) =
                    make_float4(o[mt][2 * c][2 * hf] * vref, o[mt][2 * c + 1][2 * hf] * vref,
                                o[mt][2 * c][2 * hf + 1] * vref, o[mt][2 * c + 1][2 * hf + 1] * vref);
            } else {
#pragma unroll
              for (int n = 0; n < kNT; ++n)
                *reinterpret_cast<float2*>(pp + 8 * n + 2 * tq) =
                    make_float2(o[mt][n][2 * hf], o[mt][n][2 * hf + 1]);
            }
          }
        }
    }
    if (rd_left > 0) next_unit(a, rd);
  }
  // A wait that ran out left copies in flight: let them land before the shared memory goes away.
  if (!ok && lane == 0)
    for (int i = max(used, issued - C::kStages); i < issued; ++i)
      mbar_wait_drain(&full[warp][i % C::kStages], (i / C::kStages) & 1, st);
}

// ------------------------------------------------------------------------------------
// Merge of the units cut between CTAs: block (c, y) takes the unit that begins in CTA c and ends in
// a later one, a warp one of its rows.  With parts (m_i, l_i, O_i):
//     O = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i,  m = max_i m_i.
// ------------------------------------------------------------------------------------
template <int D, bool kFp16>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeArgs a) {
  constexpr int kV = D / 32;                              // columns per lane
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, lane = lane_id();
  const int4 me = a.meta[2 * c];                          // last CTA, rows, first token, key head
  const int row0 = a.meta[2 * c + 1].x;
  const int r = blockIdx.y * 8 + warp_id();
  if (me.x < 0 || r >= me.y) return;
  const int n = me.x - c + 1;                             // parts: this CTA's and those of c + 1 .. me.x
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) {
    const long long slot = i == 0 ? 2LL * c + 1 : 2LL * (c + i);
    m = fmaxf(m, a.part_ml[(slot * a.slot_rows + r) * 2]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float neg = m == -INFINITY ? 0.f : -m;
  float l = 0.f, acc[kV] = {};
  for (int i0 = 0; i0 < n; i0 += 32) {
    float w = 0.f;
    if (i0 + lane < n) {
      const long long slot = i0 + lane == 0 ? 2LL * c + 1 : 2LL * (c + i0 + lane);
      const float* ml = a.part_ml + (slot * a.slot_rows + r) * 2;
      w = ex2(ml[0] + neg);
      l += w * ml[1];
    }
    const int k = min(32, n - i0);
#pragma unroll 8
    for (int i = 0; i < k; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const long long slot = i0 + i == 0 ? 2LL * c + 1 : 2LL * (c + i0 + i);
      const float* p = a.part_o + (slot * a.slot_rows + r) * D + lane * kV;
      if constexpr (kV == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        acc[0] += wi * x.x;
        acc[1] += wi * x.y;
        acc[2] += wi * x.z;
        acc[3] += wi * x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(p);
        acc[0] += wi * x.x;
        acc[1] += wi * x.y;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int t = (row0 + r) / a.G, g = (row0 + r) - t * a.G;
  const long long tk = me.z + t;
  const int hq = me.w * a.G + g;
  if (lane == 0) a.lse[tk * a.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2f;
  uint32_t* op = reinterpret_cast<uint32_t*>(a.o + tk * a.o_tok + hq * a.o_head + lane * kV);
#pragma unroll
  for (int i = 0; i < kV; i += 2) op[i / 2] = pack2<kFp16>(acc[i] * inv, acc[i + 1] * inv);
}

template <int D, bool kFp8, bool kFp16, int kMT>
cudaError_t launch_small(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, int ctas, cudaStream_t s) {
  auto kern = tree_small_kernel<D, kFp8, kFp16, kMT>;
  constexpr int smem = SmallCfg<D, kFp8>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<ctas, 256, smem, s>>>(tk, tv, a);
  return cudaGetLastError();
}

template <int D, bool kFp8, bool kFp16>
cudaError_t launch_small_mt(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, int ctas, cudaStream_t s) {
  return a.tile_rows == 16 ? launch_small<D, kFp8, kFp16, 1>(tk, tv, a, ctas, s)
                           : launch_small<D, kFp8, kFp16, 2>(tk, tv, a, ctas, s);
}

template <int D>
cudaError_t launch_small_d(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, bool fp8, bool fp16,
                           int ctas, cudaStream_t s) {
  if (fp8) return fp16 ? launch_small_mt<D, true, true>(tk, tv, a, ctas, s) : launch_small_mt<D, true, false>(tk, tv, a, ctas, s);
  return fp16 ? launch_small_mt<D, false, true>(tk, tv, a, ctas, s) : launch_small_mt<D, false, false>(tk, tv, a, ctas, s);
}

// Launched so that its blocks may start while the attention kernel still runs (they wait for its
// end on the device): saves most of a launch's latency.
template <int D, bool kFp16>
cudaError_t launch_merge_d(const TreeArgs& a, int ctas, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas, (a.tile_rows + 7) / 8, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, kFp16>, a);
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

// Most rows a row tile can have in a call with this many new tokens.
int most_rows(int total, int G) {
  const long long r = ((long long)total * G + 15) / 16 * 16;
  return (int)(r < kBigRows ? r : kBigRows);
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
  if (x.total == 0 || x.max_new == 0) return FA_OK;
  if (!x.q || !x.o || !x.lse || !aligned(x.q, 16) || !aligned(x.o, 16) || !aligned(x.lse, 4)) return FA_ERR_INVALID_ARG;
  for (const long long s : {(long long)x.q_token_stride, (long long)x.q_head_stride, (long long)x.o_token_stride,
                            (long long)x.o_head_stride})
    if (s < 0 || s % 8 != 0) return FA_ERR_INVALID_ARG;
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
  const bool big = unit > 32;
  a.tile_rows = big ? kBigRows : unit <= 16 ? 16 : 32;
  a.slot_rows = min(a.tile_rows, most_rows(x.total, G));
  a.chunk_shift = !big && x.cache.d * (fp8 ? 1 : 2) <= 128 ? 8 : 7;   // 32-key steps: SmallCfg

  CUtensorMap tk, tv;
  const long long rows = (long long)x.cache.pages * x.cache.Hk * x.cache.page_size;
  if (!encode_cache(&tk, x.cache.k, rows, x.cache.d, fp8 ? 1 : 2, big ? x.cache.page_size : 16, !big) ||
      !encode_cache(&tv, x.cache.v, rows, x.cache.d, fp8 ? 1 : 2, big ? x.cache.page_size : 16, !big))
    return FA_ERR_CUDA;
  // One CTA per SM, fewer where the longest possible sequences have fewer chunks.
  const long long kt = (((long long)x.cache.max_pages * x.cache.page_size - 1) >> a.chunk_shift) + 1;
  const long long rt = ((long long)x.max_new * G + a.tile_rows - 1) / a.tile_rows;
  long long most = kt * rt;
  most = most > kTreeCtas ? kTreeCtas : most * x.cache.Hk;
  most = most > kTreeCtas ? kTreeCtas : most * x.cache.B;
  const int ctas = (int)(most > kTreeCtas ? kTreeCtas : most);
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
