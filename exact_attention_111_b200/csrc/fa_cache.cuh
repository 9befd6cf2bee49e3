// fa_cache.cuh -- the paged key/value cache as the kernels see it: slot addressing, the E4M3 row
// format (quantise, expand), and the schedule of the attention over the cache, shared by its
// kernels.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fa.h"
#include "fa_internal.h"

namespace fa {

// K and V pages [pages][Hk][page_size][d], E8M0 scale codes [pages][Hk][page_size] (E4M3 only).
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  uint8_t* ks;
  uint8_t* vs;
  const int* table;      // [B, max_pages], rows table_stride apart
  int* status;           // device status word
  int pages, Hk, d, B, max_pages, table_stride;
  int page_shift;        // log2(page_size)
};

// Records a page id, length or index that the cache cannot hold; the first error wins.
__device__ __forceinline__ void flag_range(const CacheView& c) { atomicCAS(c.status, 0, kDevRange); }

// Row index (page * Hk + h) * page_size + r of key position pos of sequence b, or -1 (flagged)
// when the position lies past the table or its page id is no page.
__device__ __forceinline__ long long slot_row(const CacheView& c, int b, int h, long long pos) {
  const long long e = pos >> c.page_shift;
  if (pos < 0 || e >= c.max_pages) {
    flag_range(c);
    return -1;
  }
  const int p = c.table[(long long)b * c.table_stride + e];
  if (p < 0 || p >= c.pages) {
    flag_range(c);
    return -1;
  }
  return (((long long)p * c.Hk + h) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// The sequence that owns token tok: the last b with cu[b] <= tok < cu[b + 1], or -1.  One warp
// searches 32-ary: 2 rounds of independent loads up to 1024 sequences.
__device__ __forceinline__ int owner_of(const int* cu, int B, int tok) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B + 1;                 // count of entries cu[lo .. lo + n) <= tok, over cu[0 .. B]
  while (n > 0) {
    const int step = (n + 31) >> 5;
    const int i = lo + (lane + 1) * step - 1;
    const bool le = (lane + 1) * step <= n && cu[i] <= tok;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    lo += c * step;
    n = min(step - 1, n - c * step);
  }
  return lo >= 1 && lo <= B ? lo - 1 : -1;
}

// ------------------------------------------------------------------------------------
// E4M3 rows.  A row of d values x is stored as codes and one power-of-two scale 2^e, with e the
// smallest exponent for which max |x| <= 448 * 2^e: the largest magnitude lands in (224, 448], the
// codes are x * 2^-e (an exact product) rounded to nearest even, and code * 2^e is exact in
// bf16 (from its smallest normal value up), so reading back adds no error.  A power of two costs no precision against max/448: E4M3
// is a floating type, so a factor below 2 moves no value out of its normal range but the lowest binade.
// ------------------------------------------------------------------------------------

// E8M0 code e + 127 of a row whose largest finite magnitude is amax: with amax = 2^(E-127) (1 + M),
// e = E - 127 - 8, one more when 1 + M > 1.75 (448 = 1.75 * 2^8).
__device__ __forceinline__ int scale_code(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int s = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(s, 1);                      // at most 254 - 8 + 1 = 247
}
// 2^(code - 127), code 0 .. 254 (0: below fp32's normal range)
__device__ __forceinline__ float scale_value(uint32_t code) { return __uint_as_float(code == 0 ? 0x400000u : code << 23); }
__device__ __forceinline__ float scale_inverse(int code) { return __uint_as_float((254u - code) << 23); }

// Two fp32 to two E4M3 codes (lo = first), round to nearest even; NaN gives the NaN code.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two E4M3 codes (low 16 bits) to two fp16, exact.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// bf16 queries meet an E4M3 cache's codes in fp16 products: a row is scaled by 2^k, which brings its
// largest magnitude amax to [2^14, 2^15) (as far as k <= 112 does): the eight bits of a value are kept
// down to 2^-28 of the largest, and below that the error stays under 2^-39 of it.
__device__ __forceinline__ int row_factor(float amax) {
  const int ex = static_cast<int>(__float_as_uint(amax) >> 23);      // biased exponent
  return ex == 255 ? 0 : max(-113, min(112, 127 + 14 - ex));
}

// Probabilities enter fp16 products as 2^15 times exp(s - max), the most that fp16 holds: then they have
// its eleven bits down to 2^-29 of the largest (2^-14 without the factor), and what is below is off by at most
// 2^-40 of it.  Many keys of small probability together count in a long context, and
// without the factor those of 1.4 * 2^-24 were all 29 % off.  The row sum has the factor too, so it drops out of O; the running max is
// kept less 15, so that max + log2(sum) is the LSE as before and parts merge as before.
constexpr float kFp16Lift = 15.f;

// ------------------------------------------------------------------------------------
// Schedule of the attention over the cache.  A unit is one (sequence, key head, row tile): rows are
// the unit's (new token, query head of the group) pairs.  Its keys are cut into chunks of 128 or 256.
// All chunks of all units stand in one line -- sequences, in them key heads, in them row tiles,
// in them chunks -- and CTA c of C takes the c-th of C equal parts, whatever units it cuts.
// Every warp finds its part from the lengths on the device, so the host needs none of them.
// ------------------------------------------------------------------------------------

constexpr int kChunk = 128;      // keys of a chunk of the tensor-memory kernel (the other has 128 or 256)
constexpr int kTreeCtas = 148;   // most CTAs (one per SM)
constexpr int kBigRows = 256;    // rows of a unit of the tensor-memory kernel

struct TreeArgs {
  CacheView c;
  const uint16_t* q;             // [total, Hq, d], strides below
  uint16_t* o;                   // [total, Hq, d]
  float* lse;                    // [total, Hq], dense
  const int* cu;                 // [B + 1]
  const int* lens;               // [B]
  const unsigned long long* mask;   // [total, words] or null
  float* part_o;                 // [C, 2, slot_rows, d] partial sums of units cut between CTAs
  float* part_ml;                // [C, 2, slot_rows, 2] their running max (log2 units) and sum
  int4* meta;                    // [C, 2] a cut unit that begins in CTA c: its last CTA (-1: none), rows, first
                                 // token and key head; its first row
  long long q_tok, q_head, o_tok, o_head;   // strides in elements
  int total, Hq, G, words, max_new;
  int tile_rows;                 // rows of a row tile
  int slot_rows;                 // rows of a slot of part_o / part_ml: at least a unit's rows
  int chunk_shift;               // log2 of a chunk's keys: 7 or 8
  unsigned long long timeout_ns;
  float scale_log2;
};

// One sequence's numbers.
struct SeqView {
  int T, len, cu0;               // new tokens, prefix keys, first token
  int RT, KT;                    // row tiles per key head, chunks
};

// Reads sequence b; T = 0 where there is nothing to do or (flagged) the lengths cannot be.
__device__ __forceinline__ SeqView load_seq(const TreeArgs& a, int b, bool flag) {
  SeqView s{0, 0, 0, 0, 0};
  const int c0 = a.cu[b], c1 = a.cu[b + 1], len = a.lens[b];
  const long long T = (long long)c1 - c0, L = (long long)len + T;
  if (T == 0) return s;
  if (T < 0 || T > a.max_new || c0 < 0 || c1 > a.total || len < 0 ||
      ((L - 1) >> a.c.page_shift) >= a.c.max_pages) {
    if (flag) flag_range(a.c);
    return s;
  }
  s.T = (int)T;
  s.len = len;
  s.cu0 = c0;
  s.RT = s.T * a.G <= a.tile_rows ? 1 : (s.T * a.G - 1) / a.tile_rows + 1;     // max_new * G < 2^31
  s.KT = (int)((L - 1) >> a.chunk_shift) + 1;
  return s;
}

// A place in the line of chunks: sequence b, unit u = key head * RT + row tile, chunk kt.
struct Cursor {
  SeqView s;
  int b, u, kt;
  int h;                         // the unit's key head
  int last;                      // last key position that a row of the unit may see
};

__device__ __forceinline__ void enter_unit(const TreeArgs& a, Cursor& c) {
  c.h = c.s.RT == 1 ? c.u : c.u / c.s.RT;
  c.last = c.s.len + c.s.T - 1;
  if (a.mask == nullptr && c.s.RT > 1) {   // chain: up to the row tile's last token
    const long long end = ((long long)(c.u - c.h * c.s.RT + 1) * a.tile_rows + a.G - 1) / a.G;
    if (end < c.s.T) c.last = c.s.len + (int)end - 1;
  }
}

// The line's total and equal parts: the first `more` CTAs take each + 1 chunks, the others `each`; no part
// is empty while another has two.  Units of fewer than 2^31 chunks in all (32-bit divisions).
struct Line {
  int each, more;
  __device__ __forceinline__ int count(int cta) const { return each + (cta < more ? 1 : 0); }
  __device__ __forceinline__ int first(int cta) const { return cta * each + min(cta, more); }
  // the CTA whose part holds chunk g
  __device__ __forceinline__ int owner(int g) const {
    const int cut = more * (each + 1);
    return g < cut ? g / (each + 1) : more + (g - cut) / each;
  }
};

// This CTA's part and the place of its first chunk; one warp together.  flag: report sequences whose
// lengths cannot be.
struct Part {
  Line line;
  int lo, n;
  Cursor at;
};

__device__ __forceinline__ Part find_part(const TreeArgs& a, bool flag) {
  const int lane = threadIdx.x & 31, B = a.c.B;
  // chunks of each lane's sequence of the first 32, and of all
  SeqView s{0, 0, 0, 0, 0};
  if (lane < B) s = load_seq(a, lane, flag);
  long long n = (long long)s.RT * s.KT * a.c.Hk, total = n;
  for (int b = 32 + lane; b < B; b += 32) {
    const SeqView t = load_seq(a, b, flag);
    total += (long long)t.RT * t.KT * a.c.Hk;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  Part p{};
  if (total >= (1LL << 31)) {
    if (flag) flag_range(a.c);
    total = 0;
  }
  p.line.each = (int)total / (int)gridDim.x;
  p.line.more = (int)total - p.line.each * (int)gridDim.x;
  p.n = p.line.count(blockIdx.x);
  p.lo = p.line.first(blockIdx.x);
  if (p.n == 0) return p;
  int g = p.lo;
  for (int base = 0;;) {
    int inc = (int)n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, inc > g);
    if (hit != 0) {
      const int src = __ffs(hit) - 1;
      g -= __shfl_sync(0xffffffffu, inc - (int)n, src);
      p.at.b = base + src;
      p.at.s.T = __shfl_sync(0xffffffffu, s.T, src);
      p.at.s.len = __shfl_sync(0xffffffffu, s.len, src);
      p.at.s.cu0 = __shfl_sync(0xffffffffu, s.cu0, src);
      p.at.s.RT = __shfl_sync(0xffffffffu, s.RT, src);
      p.at.s.KT = __shfl_sync(0xffffffffu, s.KT, src);
      p.at.u = g / p.at.s.KT;
      p.at.kt = g - p.at.u * p.at.s.KT;
      enter_unit(a, p.at);
      return p;
    }
    g -= __shfl_sync(0xffffffffu, inc, 31);
    base += 32;
    s = SeqView{0, 0, 0, 0, 0};
    if (base + lane < B) s = load_seq(a, base + lane, false);
    n = (long long)s.RT * s.KT * a.c.Hk;
  }
}

// The next chunk; only called while chunks are left.
__device__ __forceinline__ void next_unit(const TreeArgs& a, Cursor& c) {
  c.kt = 0;
  if (++c.u >= c.s.RT * a.c.Hk) {
    c.u = 0;
    do {
      if (++c.b >= a.c.B) return;
      c.s = load_seq(a, c.b, false);
    } while (c.s.T == 0);
  }
  enter_unit(a, c);
}

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

template <int N>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Host side (fa_cache.cu): checks of the cache argument, and its view.
int check_cache(const fa_cache& c);
CacheView view_of(const fa_cache& c);
// fa_host.cu: what fa_last_launch_count returns, and the TMA map of a cache's rows [rows][d] in
// boxes of box_rows rows, 128-byte panels (64-byte rows for E4M3 at d = 64), swizzled: a box holds all
// panels (one after the other) or one.
void note_launches(int n);
bool encode_cache(CUtensorMap* m, const void* base, long long rows, int d, int elem, int box_rows, bool all_panels);

// Sets a kernel's dynamic shared memory once per device, and checks once that it was built with the registers
// its setmaxnreg shares assume (the increase waits until the block's launch registers cover them).
template <typename F>
cudaError_t prepare_kernel(F* kern, int smem, int regs, bool (&done)[128]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 128) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes at;
  e = cudaFuncGetAttributes(&at, kern);
  if (e != cudaSuccess) return e;
  if (at.numRegs != regs) return cudaErrorInvalidConfiguration;
  done[dev] = true;              // two threads may both get here: the same is done twice
  return cudaSuccess;
}

// The cache's and the attention's kernels may be brought onto the SMs while the kernel before them in the stream still runs:
// they are launched so, set up their barriers, and in grid_begin wait for that kernel's end and for its
// writes to be visible, before the first access to global memory; then they let the next one come.
__device__ __forceinline__ void grid_begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... A, typename... B>
cudaError_t launch_after(void (*kern)(A...), dim3 grid, int threads, size_t smem, cudaStream_t s, const B&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<A>(args)...);
}

cudaError_t launch_tree_big(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, bool fp8, bool fp16,
                            int ctas, cudaStream_t s);

}  // namespace fa
