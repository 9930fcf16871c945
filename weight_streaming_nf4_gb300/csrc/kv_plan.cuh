// kv_plan.cuh -- the layout of a cache plan (see ws_kv_plan): what
// k_kv_plan writes on the device and the append and attention kernels read.
#pragma once
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace ws {

constexpr int kPage = WS_KV_PAGE;
constexpr int kTileRows = 16;    // rows of a tile of the decode kernel, which has the sequences of up to so many
// Resident warps of the decode kernel an SM: eight with 24 KB of pages on their
// way each (D = 128), twelve with 12 KB (D = 64).
constexpr int decode_warps(int hd) { return hd == 128 ? 8 : 12; }
constexpr int kChunkRows = 256;  // rows of a tile of the chunk kernel, which has the others
constexpr int kChunkMinSteps = 12;  // steps (two pages) of a share of the chunk kernel's work, at least
// What beginning a tile costs, in steps: a share's length counts it, so that shares with many beginnings end with the
// others.  Tiles of up to half the rows, whose two slots share their steps, have an entry of their own, and their
// steps count half.  In us, four draws of inputs in turn: two prompts (1800 + 1519 rows of 40 + 8 heads behind 6000 and
// 3392 tokens), a step with three prompts of 485 to 700 rows among 30 single ones (28 + 4 heads), 24 sequences of 4 and
// of 20 rows (40 + 8 heads; 240k and 60k tokens in all), and with 14 + 2 heads of 64 the prompts and the mixed step again:
// 10 and 4 421, 165, 156, 72, 137, 89; 8 and 3 418, 164, 156, 70, 136, 85; 5 and 3 413, 164, 156, 70, 136, 83; 4 and 2
// 414, 165, 159, 75, 135, 83.
constexpr int kChunkTileCost = 5, kChunkHalfTileCost = 3;
static_assert(kChunkMinSteps > kChunkTileCost, "every share has a step");

// Rows are a sequence's (new token, query head of one kv head) pairs, token by
// token.  The decode kernel's plan is per kv head, the same for all; the chunk
// kernel's shares run over all kv heads, one after another.
struct KvHeader {
  int n_append;  // touched pages
  int n_tiles;   // decode: tiles
  int pages;     // sum of their pages
  int units;     // equal shares of those pages, one warp each
  int n_split;   // tiles cut by a unit's end
  int c_tiles;   // chunk: tiles
  int c_steps;   // sum of their steps
  int c_units;   // shares of n_kv_heads times those, equal in cost, one CTA each
  int c_split;   // (head, tile) pairs cut by a unit's end
  uint32_t sig[2];  // of the sizes that it was made for
  int pad[5];
};
// int4 arrays:
//   seq     {tokens before the call, first row of q, new tokens, 0}
//   append  {first row, page (-1: none), first place in it, rows}
//   tile    {sequence, 0, pages of the tiles before it, index among the cut ones or -1}, a sequence
//           each, one more at the end with the pages of all
//   split   two each: {first slot, pieces, first row, 0}, the sequence's entry
//   c_tile  {sequence, first row, steps of the tiles before it, their cost}, one more at the end
//   c_split two each: {first slot, pieces, first row, head}, the sequence's entry
// and
//   pre     prefix sums over the sequences {pages to append to, tiles, chunk tiles, 0}
//   unit    first tile of each unit (int)
//   c_unit  {first tile, first head, index among the cut pairs of the one that its start cuts or -1, first
//           step of the tile}, one more at the end
struct KvLayout {
  size_t seq, pre, append, tile, split, unit, c_tile, c_split, c_unit, bytes;  // byte offsets
  int64_t max_append, max_tiles, max_units, c_max_tiles, c_max_units;
  uint32_t sig[2];
};

struct KvShape {
  int64_t T;
  int n_seq, max_pages, max_new, nh, nkv, hd;
};

inline int64_t kv_chunk_tiles(const KvShape& s) {
  const int64_t live = std::min<int64_t>(s.n_seq, s.T), G = s.nh / s.nkv;
  if ((int64_t)s.max_new * G <= kTileRows) return 0;
  return s.T * G / kChunkRows + std::min<int64_t>(live, s.T * G / (kTileRows + 1));
}

inline KvLayout kv_layout(const KvShape& s) {
  KvLayout L = {};
  const int64_t live = std::min<int64_t>(s.n_seq, s.T), G = s.nh / s.nkv;
  // n rows touch (n + 62) / 64 + 1 pages at most
  L.max_append = std::min<int64_t>(std::min<int64_t>(s.T, live * (((int64_t)s.max_new + 62) / kPage + 1)),
                                   s.T / kPage + 2 * live);
  L.max_tiles = G <= kTileRows ? live : 0;
  L.max_units = std::max<int64_t>(1, (int64_t)device_sm_count() * decode_warps(s.hd) / s.nkv);
  L.c_max_tiles = kv_chunk_tiles(s);
  L.c_max_units = device_sm_count();
  size_t o = sizeof(KvHeader);
  auto take = [&](int64_t n) {
    const size_t at = o;
    o += ((size_t)n + 15) / 16 * 16;
    return at;
  };
  L.seq = take((int64_t)s.n_seq * 16);
  L.pre = take((int64_t)s.n_seq * 16);
  L.append = take(L.max_append * 16);
  L.tile = take((L.max_tiles + 1) * 16);
  L.split = take(L.max_units * 32);
  L.unit = take(L.max_units * 4);
  L.c_tile = take((L.c_max_tiles + 1) * 16);
  L.c_split = take(L.c_max_units * 32);
  L.c_unit = take((L.c_max_units + 1) * 16);
  L.bytes = o;
  uint64_t h = 0x9e3779b97f4a7c15ull;  // the sizes, mixed: no zeros, no other plan's
  for (const int64_t x : {s.T, (int64_t)s.n_seq, (int64_t)s.max_pages, (int64_t)s.max_new, (int64_t)s.nh, (int64_t)s.nkv,
                          (int64_t)s.hd, (int64_t)device_sm_count()}) {
    h = (h ^ (uint64_t)x) * 0xbf58476d1ce4e5b9ull;
    h ^= h >> 31;
  }
  L.sig[0] = (uint32_t)h | 1u;
  L.sig[1] = (uint32_t)(h >> 32);
  return L;
}
// True where the memory holds a plan of these sizes.  What reads a plan asks first: memory that was never filled, or for
// other sizes, would lead it anywhere.
WS_DEVINL bool plan_filled(const uint8_t* plan, const uint32_t (&sig)[2]) {
  const KvHeader* h = reinterpret_cast<const KvHeader*>(plan);
  return h->sig[0] == sig[0] && h->sig[1] == sig[1];
}
#ifdef WS_HAS_WAITS
// The same for a kernel; one that has to leave says so in the device error word.
WS_DEVINL bool plan_filled_or_say(const uint8_t* plan, const uint32_t (&sig)[2]) {
  const bool ok = plan_filled(plan, sig);
  if (!ok && threadIdx.x == 0) atomicOr(&g_dev_error, DERR_BAD_CONFIG);
  return ok;
}
#endif

// Unit u has places [unit_start(u), unit_start(u + 1)) of W; unit_of is its inverse.
__host__ __device__ inline int64_t unit_start(int u, int64_t W, int U) { return u * W / U; }
__host__ __device__ inline int unit_of(int64_t place, int64_t W, int U) {
  return (int)(((place + 1) * U - 1) / W);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct KvAttnArgs {
  const uint8_t *k, *v;
  const float* scale;   // [n_pages][nkv][2]
  const uint8_t* plan;
  KvLayout L;
  const int32_t* table;
  const uint16_t* q;
  uint16_t* o;
  float* lse;           // [nh][T] or NULL
  float* part_o;        // [slot][nkv][kTileRows][D] of cut tiles, divided by their sums
  float* part_l;        // [slot][nkv][kTileRows] log2 of their sums
  int64_t n_pages, sq, so, T;
  int nkv, G, max_pages;
  float sl2;            // softmax scale times log2(e)
};

// Lets a kernel have `bytes` of dynamic shared memory, once a device.
template <auto KERNEL>
inline cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// 2^x with the hardware approximation (relative error about 2^-22).
WS_DEVINL float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
WS_DEVINL uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// O's reference.  A row's sum of exponentials goes by m, its scores' maximum; what it gathers from the values by
// 2^(m + ref), ref a whole number: a page whose values' scale is 2^e enters with 2^(x - m) 2^(e - ref), so what counts
// for fp16's range is the weight times the scale.  (By the largest scale alone, a page of no weight would push the
// others out of fp16.)  `at` is the largest score of a page less m: the least reference that holds the page.  Pages whose
// scores all lie 100 or more below m do not count.
WS_DEVINL float page_ref(float at, float e) { return at > -100.0f ? ceilf(at + e) : -INFINITY; }
// The factor of 2^(x - m) for a page of exponent e, 2^margin included.
WS_DEVINL float page_factor(float e, float ref, float margin) { return e - ref > 110.0f ? 0.0f : ex2(e - ref + margin); }
// A values' scale as f 2^e: f = 1 for the powers of two that append makes, NaN for NaN; other numbers (f in (1/2, 1))
// serve too.
WS_DEVINL float scale_parts(float s, float& f) {
  const uint32_t b = __float_as_uint(s), rest = b & 0x007fffffu;
  const bool normal = b - 0x00800000u < 0x7f000000u;
  f = !normal ? s * 0x1p126f : rest ? __uint_as_float(rest | 0x3f000000u) : 1.0f;
  return normal ? (float)((int)(b >> 23) - 127 + (rest != 0)) : -126.0f;
}
// 2^e for a whole number, brought into [-126, 127].
WS_DEVINL float pow2(float e) {
  return __uint_as_float((uint32_t)((int)fminf(fmaxf(e, -126.0f), 127.0f) + 127) << 23);
}
// Two probabilities as fp16 and what that leaves, also fp16: 2^-22 of themselves, or 2^-25 where that is more.
WS_DEVINL void split_f16x2(float a, float b, uint32_t& hi, uint32_t& rest) {
  hi = pack_f16x2(a, b);
  float x, y;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}"
      : "=f"(x), "=f"(y)
      : "r"(hi));
  rest = pack_f16x2(a - x, b - y);
}
// Codes 0, 1 (lo) and 2, 3 (hi) of a word, exact in fp16.
WS_DEVINL void decode4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// Two codes of the nearest e4m3 values (ties to even); a in the low byte.
WS_DEVINL uint32_t e4m3x2(float a, float b) {
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(b), "f"(a));
  return h;
}
// The same for e5m2.
WS_DEVINL uint32_t e5m2x2(float a, float b) {
  uint16_t h;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(h) : "f"(b), "f"(a));
  return h;
}
// The values of two codes (low byte first).
WS_DEVINL void e4m3x2_values(uint32_t w, float& lo, float& hi) {
  asm("{\n .reg .b32 x;\n .reg .b16 l, h;\n cvt.rn.f16x2.e4m3x2 x, %2;\n mov.b32 {l, h}, x;\n"
      " cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}"
      : "=f"(lo), "=f"(hi)
      : "h"((uint16_t)w));
}

}  // namespace ws
