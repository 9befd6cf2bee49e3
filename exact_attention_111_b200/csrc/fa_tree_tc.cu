// fa_tree_tc.cu -- attention of new tokens over the paged cache when a key head has many rows
// (drafted trees, chunks of a prompt): the same mathematics as fa_tree.cu on tcgen05 tensor cores.
//
// A unit's row tile is 256 rows (two 128-row MMA tiles that share every K/V tile); CTA c walks its part
// of the line of chunks (fa_cache.cuh), one chunk = one 128-key tile.  Warp roles (512 threads):
//   warps 0-3, 4-7  softmax groups 0, 1: Q rows into shared memory, then one row per thread
//   warps 8-11      correction: O_q <- alpha O_q in TMEM; makes the V tiles that hold new tokens safe
//   warp  12        producer: the K/V ring by TMA, one box per page and 128-byte panel
//   warp  13        MMA issuer (one thread) and TMEM allocator
//   warps 14-15     complete the producer's warpgroup
// Tensor memory (512 columns): S0 [0,128), S1 [128,256), O0 [256,256+d), O1 [256+d,256+2d); P
// (16-bit) over the first 64 columns of its S.  Per tile u: O_q += P_q V(u-1), then S_q = Q_q K(u)^T, so
// a finished S_q(u) also says that O_q holds every earlier product.
//
// A masked product is 0 * v, which is not 0 where v is not finite.  Tiles that hold new tokens (which some
// rows see and others do not) or lie past the end are therefore read once more by the correction
// warps before their product: rows past the sequence's end become zero, and values that are not
// finite do too, noted; the epilogue then adds those to the rows that see them.
#include <climits>

#include "fa.h"
#include "fa_cache.cuh"
#include "sm100.cuh"

namespace fa {
namespace {

constexpr float kLn2f = 0.693147180559945309f;

template <int D>
struct BigCfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kPanelBytes = kTile * 128;
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kSmem = 2 * kTileBytes + 2 * kStages * kTileBytes + 1024;
  static constexpr int kOCol = 256;
  static constexpr int kCorrWarp = 8, kLoadWarp = 12, kMmaWarp = 13;
  // 512 threads x 128 registers at launch, shared out again by setmaxnreg: the shares add up to
  // exactly the launch's, so every increase is satisfied.
  static constexpr int kLaunchRegs = 128, kRegSoftmax = 176, kRegCorr = 88, kRegOther = 72;
  static_assert(2 * kRegSoftmax + kRegCorr + kRegOther <= 4 * kLaunchRegs, "register shares");
  // exp2 pairs per 8 on the FMA pipe's polynomial (as in the dense forward)
  static constexpr int kPolyOf8 = D == 64 ? 2 : 0;
};

struct BigShared {
  uint64_t q_full[2], o_full[2];
  uint64_t k_full[4], v_full[4], k_empty[4], v_empty[4], v_ok[4];
  uint64_t s_full[2], p_full[2], alpha_full[2], o_ready[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  // [group][its segments mod 2]: number + 1 of a segment where a new token's value was not finite.
  // Entry n + 2 of a group is written only after the group's softmax began segment n + 1.
  int odd[2][2];
  float alpha[2][kTile];
};

template <int N>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// A segment: the CTA's run of tiles [kt0, kt0 + n) of one unit; nu of them can be seen by some row.
struct Seg {
  SeqView s;
  int b, h, unit, row0, nrows, kt0, n, nu;
  bool from_start, to_end;
  long long g;                   // first chunk in the line
};

__device__ __forceinline__ Seg take_segment(const TreeArgs& a, Cursor& c, long long& g, int& left) {
  Seg e;
  e.s = c.s;
  e.b = c.b;
  e.h = c.h;
  e.unit = c.u;
  e.row0 = (c.u - c.h * c.s.RT) * a.tile_rows;
  e.nrows = (int)min((long long)a.tile_rows, (long long)c.s.T * a.G - e.row0);
  e.kt0 = c.kt;
  e.n = min(c.s.KT - c.kt, left);
  e.nu = max(0, min(e.n, c.last / kChunk + 1 - c.kt));
  e.from_start = c.kt == 0;
  e.to_end = c.kt + e.n == c.s.KT;
  e.g = g;
  g += e.n;
  left -= e.n;
  if (left > 0) next_unit(a, c);
  return e;
}

// Whether tile kt holds new tokens or reaches past them.
__device__ __forceinline__ bool tail_tile(const Seg& e, int kt) { return (kt + 1) * kChunk > e.s.len; }

// Bits of the 32 keys from new token n0 on (negative: prefix) that token t of the sequence sees.
__device__ __forceinline__ uint32_t visible32(const TreeArgs& a, const SeqView& s, int t, int n0) {
  if (n0 <= -32) return 0xFFFFFFFFu;
  if (n0 >= s.T) return 0u;
  uint32_t v;
  if (a.mask == nullptr) {
    const int k = t + 1 - n0;
    v = k >= 32 ? 0xFFFFFFFFu : k <= 0 ? 0u : (1u << k) - 1u;
  } else {
    const unsigned long long* row = a.mask + (long long)(s.cu0 + t) * a.words;
    if (n0 < 0) {
      v = (uint32_t)(row[0] << -n0) | ((1u << -n0) - 1u);
    } else {
      const int w = n0 >> 6, sh = n0 & 63;
      unsigned long long x = w < a.words ? row[w] >> sh : 0ull;
      if (sh > 32 && w + 1 < a.words) x |= row[w + 1] << (64 - sh);
      v = (uint32_t)x;
    }
  }
  const int k = s.T - n0;        // new tokens end here
  return k < 32 ? v & ((1u << k) - 1u) : v;
}

template <int D, bool kFp16>
__global__ void __launch_bounds__(512, 1)
    tree_big_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const TreeArgs a) {
  using C = BigCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ BigShared sh;
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  uint8_t* sQ = smem_raw + pad;
  uint8_t* sK = sQ + 2 * C::kTileBytes;
  uint8_t* sV = sK + C::kStages * C::kTileBytes;
  const int warp = warp_id(), lane = lane_id();
  const DevStatus st{a.c.status, a.timeout_ns};
  volatile int* abort_flag = &sh.abort_flag;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh.k_full[s], 1);
      mbar_init(&sh.v_full[s], 1);
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
    mbar_init(&sh.mma_done, 1);
    sh.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
  }
  const long long total = total_chunks(a, blockIdx.x == 0 && warp == 0);
  const Part part = part_of(total, blockIdx.x, gridDim.x);
  if (threadIdx.x == 0) a.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
  Cursor cur{};
  if (part.n > 0) cur = locate(a, part.lo);
  long long g = part.lo;
  int left = part.n;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;

  if (warp >= C::kLoadWarp) {
    reg_dec<C::kRegOther>();
    if (warp == C::kLoadWarp) {
      // ---------------------------------------------------------------- producer
      const int R = 1 << a.c.page_shift;                  // rows per box: one page
      const int boxes = kTile / R;
      int nk = 0, nv = 0;                                 // tiles whose copy was started
      bool ok = true;
      if (lane == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
      }
      while (left > 0 && ok) {
        const Seg e = take_segment(a, cur, g, left);
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
      if (lane == 0) {
        const uint32_t idesc_s = idesc_f16(128, 128, kFp16, false, false);
        const uint32_t idesc_pv = idesc_f16(128, D, kFp16, false, true);
        const uint32_t aQ = smem_addr(sQ), aK = smem_addr(sK), aV = smem_addr(sV);
        int nt = 0;                                       // tiles before this segment
        int np[2] = {0, 0};                               // P tiles consumed
        uint32_t tails = 0;                               // bit s: parity of stage s's safe V tiles
        uint32_t nseg[2] = {0, 0};
        bool ok = true;
        while (left > 0 && ok) {
          const Seg e = take_segment(a, cur, g, left);
          const int nq = e.nrows > kTile ? 2 : 1;
          for (int u = 0; u <= e.nu && ok && e.nu > 0; ++u) {
            const int tp = nt + u - 1, tc = nt + u;
            const int sp = (tp + C::kStages) % C::kStages, sc = tc % C::kStages;
            bool v_ready = false, k_ready = false;
            auto pv = [&](int q) -> bool {
              if (u == 0 || q >= nq) return true;
              if (!v_ready) {
                if (!mbar_wait(&sh.v_full[sp], (tp / C::kStages) & 1, abort_flag, st)) return false;
                if (tail_tile(e, e.kt0 + u - 1)) {
                  if (!mbar_wait(&sh.v_ok[sp], (tails >> sp) & 1u, abort_flag, st)) return false;
                  tails ^= 1u << sp;
                }
                v_ready = true;
              }
              if (!mbar_wait(&sh.p_full[q], np[q] & 1, abort_flag, st)) return false;
              if (!mbar_wait(&sh.o_ready[q], np[q] & 1, abort_flag, st)) return false;
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk) {
                const uint64_t bdesc = smem_desc_sw128(aV + sp * C::kTileBytes + kk * 2048, C::kPanelBytes, 1024);
                mma_ts(tmem + C::kOCol + q * D, tmem + q * 128 + kk * 8, bdesc, idesc_pv, (u > 1 || kk > 0) ? 1u : 0u);
              }
              ++np[q];
              return true;
            };
            auto sq = [&](int q) -> bool {
              if (u == e.nu || q >= nq) return true;
              if (!k_ready) {
                if (!mbar_wait(&sh.k_full[sc], (tc / C::kStages) & 1, abort_flag, st)) return false;
                k_ready = true;
              }
              if (u == 0) {
                if (!mbar_wait(&sh.q_full[q], nseg[q] & 1, abort_flag, st)) return false;
                ++nseg[q];
              }
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t koff = (kk >> 2) * C::kPanelBytes + (kk & 3) * 32;
                const uint64_t adesc = smem_desc_sw128(aQ + q * C::kTileBytes + koff, 16, 1024);
                const uint64_t bdesc = smem_desc_sw128(aK + sc * C::kTileBytes + koff, 16, 1024);
                mma_ss(tmem + q * 128, adesc, bdesc, idesc_s, kk > 0 ? 1u : 0u);
              }
              tc_commit(&sh.s_full[q]);
              return true;
            };
            ok = pv(0) && sq(0) && pv(1);
            if (u > 0 && ok) tc_commit(&sh.v_empty[sp]);
            ok = ok && sq(1);
            if (u < e.nu && ok) tc_commit(&sh.k_empty[sc]);
          }
          nt += e.nu;
          if (ok && e.nu > 0)
            for (int q = 0; q < nq; ++q) tc_commit(&sh.o_full[q]);   // O_q holds every product
        }
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
    while (left > 0 && ok) {
      const Seg e = take_segment(a, cur, g, left);
      const int nq = e.nrows > kTile ? 2 : 1;
      for (int u = 0; u < e.nu && ok; ++u) {
        const int kt = e.kt0 + u;
        if (tail_tile(e, kt)) {
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
            uint32_t* w = &x.x;
            bool odd = past;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              constexpr uint32_t ex = kFp16 ? 0x7C00u : 0x7F80u;
              if ((w[i] & ex) == ex) { w[i] &= 0xFFFF0000u; odd = true; }
              if (((w[i] >> 16) & ex) == ex) { w[i] &= 0xFFFFu; odd = true; }
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
            tc_fence_after();
            const uint32_t tO = tmem + C::kOCol + q * D + lane_off;
#pragma unroll
            for (int cc = 0; cc < D; cc += 32) {
              uint32_t o[32];
              tmem_ld32_sync(tO + cc, o);
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 x = mul2(make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), make_float2(al, al));
                o[i] = __float_as_uint(x.x);
                o[i + 1] = __float_as_uint(x.y);
              }
              tmem_st32(tO + cc, o);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          mbar_arrive(&sh.o_ready[q]);
          ++cq[q];
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
    const float sl2 = a.scale_log2;
    int cs = 0, nseg = 0;
    bool ok = true;
    while (left > 0 && ok) {
      const Seg e = take_segment(a, cur, g, left);
      if (q == 1 && e.nrows <= kTile) continue;           // this group's tile has no rows
      const int r = q * kTile + rl;                       // row of the unit
      const bool live = r < e.nrows;
      const int R = e.row0 + (live ? r : 0);
      const int t = R / a.G, hq = e.h * a.G + (R - t * a.G);
      if (e.nu > 0) {
        // Q row into the swizzled tile (rows without a token: zeros)
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (e.s.cu0 + t) * a.q_tok + hq * a.q_head);
        uint8_t* dst = sQ + q * C::kTileBytes + rl * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 x = live ? src[c] : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(dst + (c >> 3) * C::kPanelBytes + (((c & 7) ^ (rl & 7)) << 4)) = x;
        }
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(&sh.q_full[q]);
      }
      float m = -INFINITY, l = 0.f;
      for (int u = 0; u < e.nu; ++u) {
        const int kt = e.kt0 + u;
        ok = mbar_wait(&sh.s_full[q], cs & 1, abort_flag, st);
        if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
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
        const float mx2 = row_max128(s) * sl2;
        float alpha = 1.f;
        if (mx2 > m) {
          alpha = ex2(m - mx2);                           // 0 when m = -inf
          m = mx2;
        }
        sh.alpha[q][rl] = alpha;
        mbar_arrive(&sh.alpha_full[q]);
        const float mneg = (m == -INFINITY) ? 0.f : -m;
        const float2 sl2v = make_float2(sl2, sl2), mnegv = make_float2(mneg, mneg);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 x = fma2(make_float2(s[32 * h + 2 * i], s[32 * h + 2 * i + 1]), sl2v, mnegv);
            const float2 p = (((16 * h + i) & 7) < C::kPolyOf8) ? exp2_poly2(x) : make_float2(ex2(x.x), ex2(x.y));
            acc[i & 3] = add2(acc[i & 3], p);
            pk[i] = pack2<kFp16>(p.x, p.y);               // at most half a 16-bit step; the sum keeps 32 bits
          }
          tmem_st16(tS + 16 * h, pk);
        }
        const float2 sum = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
        l = l * alpha + (sum.x + sum.y);
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
      if (q == 0 && rl == 0 && e.from_start && !e.to_end)
        a.meta[blockIdx.x] = make_int4(e.b, e.unit, owner_cta(total, e.g + e.s.KT - 1, gridDim.x), 0);
      const bool odd = e.nu > 0 && *reinterpret_cast<volatile int*>(&sh.odd[q][(nseg - 1) & 1]) == nseg;
      const float inv = l == 0.f ? 0.f : 1.f / l;
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
          tmem_ld32_sync(tO + cc, o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        if (!live) continue;
        if (odd) {                                        // rare: see the top of the file
          const int j1 = min(e.s.T, (e.kt0 + e.nu) * kChunk - e.s.len);
          for (int j = max(0, e.kt0 * kChunk - e.s.len); j < j1; ++j) {
            if (!(visible32(a, e.s, t, j) & 1u)) continue;
            const long long row = slot_row(a.c, e.b, e.h, (long long)e.s.len + j);
            if (row < 0) continue;
            const uint16_t* v = reinterpret_cast<const uint16_t*>(a.c.v) + row * D + cc;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              constexpr uint32_t ex = kFp16 ? 0x7C00u : 0x7F80u;
              const uint32_t w = v[i];
              if ((w & ex) == ex) o[i] = __float_as_uint(__uint_as_float(o[i]) + unpack2<kFp16>(w).x);
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
          uint4* dst = reinterpret_cast<uint4*>(a.part_o + ((long long)slot * a.slot_rows + r) * D + cc);
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
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

template <int D, bool kFp16>
cudaError_t launch_big(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, int ctas, cudaStream_t s) {
  using C = BigCfg<D>;
  auto kern = tree_big_kernel<D, kFp16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  // setmaxnreg.inc waits until the block's launch registers cover every warpgroup's share: refuse a
  // build whose register count differs from the one the shares assume.
  static int regs = 0;
  if (regs == 0) {
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, kern);
    if (e != cudaSuccess) return e;
    regs = at.numRegs;
  }
  if (regs != C::kLaunchRegs) return cudaErrorInvalidConfiguration;
  kern<<<ctas, 512, C::kSmem, s>>>(tk, tv, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_big(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, bool fp16, int ctas,
                            cudaStream_t s) {
  if (a.c.d == 128) return fp16 ? launch_big<128, true>(tk, tv, a, ctas, s) : launch_big<128, false>(tk, tv, a, ctas, s);
  return fp16 ? launch_big<64, true>(tk, tv, a, ctas, s) : launch_big<64, false>(tk, tv, a, ctas, s);
}

}  // namespace fa
