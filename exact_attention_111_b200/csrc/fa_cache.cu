// fa_cache.cu -- the paged key/value cache: rows written (and quantised) behind what a sequence
// holds, read back as dense tensors, and the accepted rows of a drafted tree moved up; with their
// C entry points (include/fa.h).  All three move bytes once and are bound by them (HBM), or by
// the latency of one launch and its dependent loads (length -> page id -> row) when small.
#include <cmath>
#include <climits>

#include "fa.h"
#include "fa_cache.cuh"
#include "sm100.cuh"

namespace fa {

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ------------------------------------------------------------------------------------
// Append.  One warp takes one new token and, kSteps times, 32 / kLanes of its key heads, K and V: a lane
// holds 8 elements (16 bytes) of K and V rows, whose loads are in flight while the token's sequence,
// position and page are looked up (four or five dependent loads).
// ------------------------------------------------------------------------------------

struct AppendArgs {
  CacheView c;
  const uint16_t* k;      // [total, Hk, d], strides in elements
  const uint16_t* v;
  long long k_tok, k_head, v_tok, v_head;
  const int* cu;
  const int* lens;
  int total, groups;      // groups of heads per token
};

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight 16-bit values of a row to eight E4M3 codes; the row is spread over kLanes lanes.  Magnitudes
// are compared as 16-bit integers (the order of the bits is the order of the values, infinities and NaN
// last), two at a time (14.8k tokens of 8 heads of 128: 18 us in a captured graph, 25 with every value checked and
// compared in 32 bits; the bytes alone take 14).
template <bool kFp16, int kLanes>
__device__ __forceinline__ uint2 quantise8(const uint4& w, int& code) {
  // A magnitude that E4M3 would round up past the source type's largest value is taken down to
  // the last one it does not (15/16 of the top binade), so that every stored value is finite
  // when it is read back in that type.  E4M3 holds no infinity: infinities become NaN, like NaN.
  constexpr float kTop = kFp16 ? 61440.f : 0x1.Ep127f;
  constexpr uint32_t kTopBits = kFp16 ? 0x7B80u : 0x7F70u;
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
  uint32_t top = max_u16x2(max_u16x2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), max_u16x2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, o));
  top = max(top & 0xFFFFu, top >> 16);
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<kFp16>(ws[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
  float amax = unpack2<kFp16>(top).x;
  if (__any_sync(0xffffffffu, top > kTopBits)) {    // rare: some value is not finite, or above kTop
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool finite = fabsf(x[i]) < INFINITY;
      x[i] = finite ? fminf(fmaxf(x[i], -kTop), kTop) : __int_as_float(0x7FFFFFFF);
      amax = fmaxf(amax, finite ? fabsf(x[i]) : 0.f);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  }
  code = scale_code(amax);
  const float inv = scale_inverse(code);
  uint2 r;
  r.x = e4m3x2(x[0] * inv, x[1] * inv) | (e4m3x2(x[2] * inv, x[3] * inv) << 16);
  r.y = e4m3x2(x[4] * inv, x[5] * inv) | (e4m3x2(x[6] * inv, x[7] * inv) << 16);
  return r;
}

template <int D, bool kFp8, bool kFp16, int kSteps>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
  grid_begin();
  const int lane = lane_id();
  const long long w = (long long)blockIdx.x * 8 + warp_id();
  const int tok = (int)(w / a.groups);
  if (tok >= a.total) return;
  const int h0 = (int)(w - (long long)tok * a.groups) * kHeads * kSteps + lane / kLanes;
  const int col = (lane % kLanes) * 8;
  uint4 xk[kSteps], xv[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    xk[i] = xv[i] = make_uint4(0, 0, 0, 0);
    const int h = h0 + i * kHeads;
    if (h < a.c.Hk) {
      xk[i] = *reinterpret_cast<const uint4*>(a.k + tok * a.k_tok + h * a.k_head + col);
      xv[i] = *reinterpret_cast<const uint4*>(a.v + tok * a.v_tok + h * a.v_head + col);
    }
  }
  if (w == 0) {                                     // one warp looks the whole list of bounds over
    bool bad = a.cu[0] < 0 || a.cu[a.c.B] > a.total;
    for (int i = lane; i < a.c.B; i += 32) bad |= a.cu[i] > a.cu[i + 1];
    if (bad) flag_range(a.c);
  }
  const int b = owner_of(a.cu, a.c.B, tok);
  if (b < 0) return;                                // past the last sequence: not a token
  const int len = a.lens[b], c0 = a.cu[b], c1 = a.cu[b + 1];
  // (a list that decreases may have led anywhere)
  const bool bounds = c0 >= 0 && c0 <= tok && tok < c1 && c1 <= a.total;
  const long long row = len < 0 || !bounds ? -1 : slot_row(a.c, b, 0, (long long)len + (tok - c0));
  if (row < 0) {
    flag_range(a.c);
    return;                                         // the whole warp: one token
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int h = h0 + i * kHeads;
    const bool live = h < a.c.Hk;
    const long long r = row + ((long long)(live ? h : 0) << a.c.page_shift);
    if constexpr (kFp8) {
      int sk, sv;
      const uint2 ck = quantise8<kFp16, kLanes>(xk[i], sk), cv = quantise8<kFp16, kLanes>(xv[i], sv);
      if (live) {
        *reinterpret_cast<uint2*>(a.c.k + r * D + col) = ck;
        *reinterpret_cast<uint2*>(a.c.v + r * D + col) = cv;
        if (col == 0) {
          a.c.ks[r] = (uint8_t)sk;
          a.c.vs[r] = (uint8_t)sv;
        }
      }
    } else if (live) {
      *reinterpret_cast<uint4*>(a.c.k + (r * D + col) * 2) = xk[i];
      *reinterpret_cast<uint4*>(a.c.v + (r * D + col) * 2) = xv[i];
    }
  }
}

template <int D, bool kFp8, bool kFp16>
cudaError_t launch_append(const AppendArgs& a, unsigned blocks, int steps, cudaStream_t s) {
  if constexpr (kFp8) {
    if (steps == 4) return launch_after(append_kernel<D, kFp8, kFp16, 4>, dim3(blocks), 256, 0, s, a);
  }
  return launch_after(append_kernel<D, kFp8, kFp16, 1>, dim3(blocks), 256, 0, s, a);
}

// ------------------------------------------------------------------------------------
// Read back: [B, Hk, N, d] 16-bit, zeros past a sequence's end.  Rows of one page and head are
// contiguous on both sides, so a block walks kReadRows positions of one (b, h), four or eight rows of K and
// V in flight a thread, with 16-byte stores.  Bound by HBM: four prompts of up to 4096 positions, 8 heads
// of 128, E4M3 to bf16, 16.5 us in a captured graph (5.8 TB/s of the bytes it needs, 90 % of a copy), 19.0 in a
// stream of eager calls; 16 sequences of up to 1024, 16 heads of 64, fp16, 14.6 and 17.9 us.
// ------------------------------------------------------------------------------------

struct ReadArgs {
  CacheView c;
  uint16_t* k;
  uint16_t* v;
  const int* lens;
  int N, tiles;
};

template <bool kFp16>
__device__ __forceinline__ uint4 expand8(uint2 w, float s) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = i < 2 ? w.x >> (16 * i) : w.y >> (16 * (i - 2));
    const float2 f = unpack2<true>(e4m3_to_f16x2(two & 0xFFFFu));
    r[i] = pack2<kFp16>(f.x * s, f.y * s);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

constexpr int kReadRows = 64;

template <int D, bool kFp8, bool kFp16>
__global__ void __launch_bounds__(256) read_kernel(const ReadArgs a) {
  constexpr int kLanes = D / 8, kPass = 256 / kLanes;      // rows per pass of the block
  grid_begin();
  const int tile = blockIdx.x % a.tiles;
  const int bh = blockIdx.x / a.tiles;
  const int b = bh / a.c.Hk, h = bh - b * a.c.Hk;
  const int col = (threadIdx.x % kLanes) * 8;
  const int len = a.lens[b];
  if (len < 0) {
    if (threadIdx.x == 0) flag_range(a.c);
    return;
  }
  const int n0 = tile * kReadRows + threadIdx.x / kLanes;
#pragma unroll
  for (int i = 0; i < kReadRows / kPass; ++i) {
    const int n = n0 + i * kPass;
    if (n >= a.N) break;
    uint4 xk = make_uint4(0, 0, 0, 0), xv = xk;
    const long long r = n < len ? slot_row(a.c, b, h, n) : -1;
    if (r >= 0) {
      if constexpr (kFp8) {
        const uint2 ck = *reinterpret_cast<const uint2*>(a.c.k + r * D + col);
        const uint2 cv = *reinterpret_cast<const uint2*>(a.c.v + r * D + col);
        xk = expand8<kFp16>(ck, scale_value(a.c.ks[r]));
        xv = expand8<kFp16>(cv, scale_value(a.c.vs[r]));
      } else {
        xk = *reinterpret_cast<const uint4*>(a.c.k + (r * D + col) * 2);
        xv = *reinterpret_cast<const uint4*>(a.c.v + (r * D + col) * 2);
      }
    }
    const long long at = ((long long)bh * a.N + n) * D + col;
    *reinterpret_cast<uint4*>(a.k + at) = xk;
    *reinterpret_cast<uint4*>(a.v + at) = xv;
  }
}

// ------------------------------------------------------------------------------------
// Keep: row lens[b] + kept[b][i] moves to row lens[b] + i, for i = 0 .. counts[b] - 1.  kept is
// strictly increasing, so kept[i] >= i and a row is never overwritten before it is read when the
// moves run in order; one warp makes all of one (b, h)'s moves of K, another those of V.  The rows of a
// step (2 to 8) are all read before the first is written.  Bound by latency: counts, list, page ids and
// rows are loads that depend on one another (64 trees, up to 7 rows kept, 8 heads of 128: 4.1 us).
// ------------------------------------------------------------------------------------

struct KeepArgs {
  CacheView c;
  const int* lens;
  const int* kept;        // [B, width]
  const int* counts;      // [B]
  int width;
};

template <int kRowBytes, bool kFp8>
__global__ void __launch_bounds__(128) keep_kernel(const KeepArgs a) {
  constexpr int kLanes = kRowBytes / 16, kRows = 32 / kLanes;
  grid_begin();
  const int lane = lane_id();
  const long long w = (long long)blockIdx.x * 4 + warp_id();
  const long long bh = w >> 1;
  if (bh >= (long long)a.c.B * a.c.Hk) return;
  const int b = (int)(bh / a.c.Hk), h = (int)(bh - (long long)b * a.c.Hk);
  uint8_t* base = (w & 1) ? a.c.v : a.c.k;
  uint8_t* scales = (w & 1) ? a.c.vs : a.c.ks;
  const int n = a.counts[b], len = a.lens[b];
  const int* kept = a.kept + (long long)b * a.width;
  // every move is checked before the first is made
  bool bad = n < 0 || n > a.width || len < 0;
  if (!bad) {
    for (int i = lane; i < n; i += 32) bad |= kept[i] <= (i > 0 ? kept[i - 1] : -1);
    if (n > 0) bad |= ((long long)len + kept[n - 1]) >> a.c.page_shift >= a.c.max_pages;
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) flag_range(a.c);
    return;
  }
  const int sub = lane / kLanes, part = (lane % kLanes) * 16;
  for (int i0 = 0; i0 < n; i0 += kRows) {
    const int i = i0 + sub;
    long long src = -1, dst = -1;
    if (i < n && kept[i] != i) {
      src = slot_row(a.c, b, h, (long long)len + kept[i]);
      dst = slot_row(a.c, b, h, (long long)len + i);
    }
    const bool go = src >= 0 && dst >= 0;
    uint4 x = make_uint4(0, 0, 0, 0);
    uint8_t s = 0;
    if (go) {
      x = *reinterpret_cast<const uint4*>(base + src * kRowBytes + part);
      if (kFp8 && part == 0) s = scales[src];
    }
    __syncwarp();                                   // all of this step's rows are read
    if (go) {
      *reinterpret_cast<uint4*>(base + dst * kRowBytes + part) = x;
      if (kFp8 && part == 0) scales[dst] = s;
    }
    __syncwarp();
  }
}

template <typename F>
int launched(F&& f) {
  return f() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Strides of a [tokens, heads, d] view: 16-byte rows, and no overlap is asked of the caller.
bool strides_ok(long long tok, long long head) { return tok >= 0 && head >= 0 && tok % 8 == 0 && head % 8 == 0; }

}  // namespace

int check_cache(const fa_cache& c) {
  if (c.B < 1 || c.Hk < 1 || c.pages < 1 || c.max_pages < 1 || c.table_stride < c.max_pages) return FA_ERR_INVALID_ARG;
  if (c.d != 64 && c.d != 128) return FA_ERR_UNSUPPORTED;
  if (c.dtype != FA_BF16 && c.dtype != FA_FP16 && c.dtype != FA_E4M3) return FA_ERR_UNSUPPORTED;
  if (c.page_size != 16 && c.page_size != 32 && c.page_size != 64 && c.page_size != 128) return FA_ERR_UNSUPPORTED;
  // row indexes are 32-bit coordinates of the copies
  if ((long long)c.pages * c.Hk > INT_MAX / c.page_size) return FA_ERR_UNSUPPORTED;
  if ((long long)c.max_pages * c.page_size > INT_MAX) return FA_ERR_UNSUPPORTED;
  if (!c.k || !c.v || !c.page_table) return FA_ERR_INVALID_ARG;
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.page_table, 4)) return FA_ERR_INVALID_ARG;
  if (c.dtype == FA_E4M3 && (!c.k_scale || !c.v_scale || !aligned(c.k_scale, 16) || !aligned(c.v_scale, 16)))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

CacheView view_of(const fa_cache& c) {
  CacheView v{};
  v.k = static_cast<uint8_t*>(c.k);
  v.v = static_cast<uint8_t*>(c.v);
  v.ks = c.k_scale;
  v.vs = c.v_scale;
  v.table = c.page_table;
  v.pages = c.pages;
  v.Hk = c.Hk;
  v.d = c.d;
  v.B = c.B;
  v.max_pages = c.max_pages;
  v.table_stride = c.table_stride;
  v.page_shift = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
  v.status = device_status_word();
  return v;
}

}  // namespace fa

using namespace fa;

extern "C" {

int fa_cache_append(const fa_cache_append_args* p) {
  if (p == nullptr) return FA_ERR_INVALID_ARG;
  const fa_cache_append_args& x = *p;
  int rc = check_cache(x.cache);
  if (rc != FA_OK) return rc;
  if (x.dtype != FA_BF16 && x.dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  if (x.cache.dtype != FA_E4M3 && x.cache.dtype != x.dtype) return FA_ERR_UNSUPPORTED;
  if (x.total < 0) return FA_ERR_INVALID_ARG;
  if (!x.cu_new || !x.lens || !aligned(x.cu_new, 4) || !aligned(x.lens, 4)) return FA_ERR_INVALID_ARG;
  if (x.total == 0) return FA_OK;
  if (!x.k_new || !x.v_new || !aligned(x.k_new, 16) || !aligned(x.v_new, 16)) return FA_ERR_INVALID_ARG;
  if (!strides_ok(x.k_token_stride, x.k_head_stride) || !strides_ok(x.v_token_stride, x.v_head_stride))
    return FA_ERR_INVALID_ARG;
  AppendArgs a{};
  int heads = 32 / (x.cache.d / 8);
  // A prompt into E4M3: four steps a warp, so that the lookup is paid for 4 KB instead of 1 KB, where three quarters of
  // the steps have a head.  Four against one, us: 16384 tokens of 8 heads of 128 23.9 : 27.3, of 6 (three of four)
  // 21.9 : 21.9, twice as many 36.2 : 38.2; of 4 (two of four) 19.8 : 16.4; 4096 tokens of 8 10.9 : 10.2.  A 16-bit cache
  // (no arithmetic) takes the same time either way, within 3 %.
  const bool fp8 = x.cache.dtype == FA_E4M3;
  const int one = (x.cache.Hk + heads - 1) / heads, four = (one + 3) / 4;      // steps for all heads; warps of four
  const int steps = fp8 && (long long)x.total * x.cache.Hk * x.cache.d >= 3LL << 22 && 4LL * one >= 12LL * four ? 4 : 1;
  heads *= steps;
  a.groups = (x.cache.Hk + heads - 1) / heads;
  const long long blocks = ((long long)x.total * a.groups + 7) / 8;
  if (blocks > INT_MAX) return FA_ERR_UNSUPPORTED;
  a.c = view_of(x.cache);
  if (!a.c.status) return FA_ERR_CUDA;
  a.k = static_cast<const uint16_t*>(x.k_new);
  a.v = static_cast<const uint16_t*>(x.v_new);
  a.k_tok = x.k_token_stride; a.k_head = x.k_head_stride;
  a.v_tok = x.v_token_stride; a.v_head = x.v_head_stride;
  a.cu = x.cu_new;
  a.lens = x.lens;
  a.total = x.total;
  const cudaStream_t s = static_cast<cudaStream_t>(x.stream);
  const bool fp16 = x.dtype == FA_FP16;
  const unsigned g = (unsigned)blocks;
  return launched([&]() -> cudaError_t {
    if (x.cache.d == 128) {
      if (!fp8) return launch_append<128, false, false>(a, g, steps, s);
      else if (fp16) return launch_append<128, true, true>(a, g, steps, s);
      else return launch_append<128, true, false>(a, g, steps, s);
    } else {
      if (!fp8) return launch_append<64, false, false>(a, g, steps, s);
      else if (fp16) return launch_append<64, true, true>(a, g, steps, s);
      else return launch_append<64, true, false>(a, g, steps, s);
    }
  });
}

int fa_cache_read(const fa_cache_read_args* p) {
  if (p == nullptr) return FA_ERR_INVALID_ARG;
  const fa_cache_read_args& x = *p;
  int rc = check_cache(x.cache);
  if (rc != FA_OK) return rc;
  if (x.dtype != FA_BF16 && x.dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  if (x.cache.dtype != FA_E4M3 && x.cache.dtype != x.dtype) return FA_ERR_UNSUPPORTED;
  if (x.N < 0 || !x.lens || !aligned(x.lens, 4)) return FA_ERR_INVALID_ARG;
  if (x.N == 0) return FA_OK;
  if (!x.k_out || !x.v_out || !aligned(x.k_out, 16) || !aligned(x.v_out, 16)) return FA_ERR_INVALID_ARG;
  ReadArgs a{};
  a.tiles = (x.N - 1) / kReadRows + 1;
  const long long blocks = (long long)x.cache.B * x.cache.Hk * a.tiles;
  if ((long long)x.cache.B * x.cache.Hk > INT_MAX || blocks > INT_MAX) return FA_ERR_UNSUPPORTED;
  a.c = view_of(x.cache);
  if (!a.c.status) return FA_ERR_CUDA;
  a.k = static_cast<uint16_t*>(x.k_out);
  a.v = static_cast<uint16_t*>(x.v_out);
  a.lens = x.lens;
  a.N = x.N;
  const cudaStream_t s = static_cast<cudaStream_t>(x.stream);
  const bool fp8 = x.cache.dtype == FA_E4M3, fp16 = x.dtype == FA_FP16;
  const unsigned g = (unsigned)blocks;
  return launched([&]() -> cudaError_t {
    if (x.cache.d == 128) {
      if (!fp8) return launch_after(read_kernel<128, false, false>, dim3(g), 256, 0, s, a);
      else if (fp16) return launch_after(read_kernel<128, true, true>, dim3(g), 256, 0, s, a);
      else return launch_after(read_kernel<128, true, false>, dim3(g), 256, 0, s, a);
    } else {
      if (!fp8) return launch_after(read_kernel<64, false, false>, dim3(g), 256, 0, s, a);
      else if (fp16) return launch_after(read_kernel<64, true, true>, dim3(g), 256, 0, s, a);
      else return launch_after(read_kernel<64, true, false>, dim3(g), 256, 0, s, a);
    }
  });
}

int fa_cache_keep(const fa_cache_keep_args* p) {
  if (p == nullptr) return FA_ERR_INVALID_ARG;
  const fa_cache_keep_args& x = *p;
  int rc = check_cache(x.cache);
  if (rc != FA_OK) return rc;
  if (x.width < 0 || !x.lens || !aligned(x.lens, 4)) return FA_ERR_INVALID_ARG;
  if (!x.counts || !aligned(x.counts, 4)) return FA_ERR_INVALID_ARG;
  if (x.width == 0) return FA_OK;
  if (!x.kept || !aligned(x.kept, 4)) return FA_ERR_INVALID_ARG;
  const long long blocks = ((long long)x.cache.B * x.cache.Hk * 2 + 3) / 4;
  if (blocks > INT_MAX) return FA_ERR_UNSUPPORTED;
  KeepArgs a{};
  a.c = view_of(x.cache);
  if (!a.c.status) return FA_ERR_CUDA;
  a.lens = x.lens;
  a.kept = x.kept;
  a.counts = x.counts;
  a.width = x.width;
  const cudaStream_t s = static_cast<cudaStream_t>(x.stream);
  const unsigned g = (unsigned)blocks;
  return launched([&]() -> cudaError_t {
    if (x.cache.dtype == FA_E4M3) {
      if (x.cache.d == 128) return launch_after(keep_kernel<128, true>, dim3(g), 128, 0, s, a);
      else return launch_after(keep_kernel<64, true>, dim3(g), 128, 0, s, a);
    } else {
      if (x.cache.d == 128) return launch_after(keep_kernel<256, false>, dim3(g), 128, 0, s, a);
      else return launch_after(keep_kernel<128, false>, dim3(g), 128, 0, s, a);
    }
  });
}

}  // extern "C"
