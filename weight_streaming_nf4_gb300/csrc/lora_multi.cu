// lora_multi.cu -- low-rank adapters of many requests beside one frozen NF4
// linear: rows sorted by adapter, the skinny products U = (mask . x) A_a^T and
// G = dY B_a, the weight gradients of every adapter, and the C entry points of
// the forward and backward.  Every reduction runs in a fixed order.
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "kernels.h"
#include "nf4_decode.cuh"

namespace ws {

namespace {

constexpr int kR = 16;            // adapter rank
constexpr int kTileRows = 64;     // rows of one skinny-product tile
constexpr int kPlanThreads = 1024;

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }
bool al16p(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ------------------------------------------------------------------------ the batch's plan
// Sections of the plan buffer (int32 words): header {tiles, slots}, the adapter
// of each row (-1: none), the rows sorted by adapter (stable; rows without one
// last), each adapter's first position in that order (n + 1 entries: the last
// is where the rows without an adapter begin), tiles {adapter, first position,
// rows, 0} of at most kTileRows rows of one adapter; and for the tensor-core
// steps of the GEMM each row's slot and, for each of its tile rows, the
// adapters of its slots (in order of their first row; -1: none).  slots: the
// most adapters of any tile row, or -1 if one has more than kMultiSlots.
struct PlanLayout {
  int64_t row, perm, off, tile, slot, tile_ad, words;
  int64_t max_tiles;
};
PlanLayout plan_layout(int64_t M, int64_t n) {
  PlanLayout L{};
  auto up4 = [](int64_t x) { return (x + 3) & ~int64_t(3); };
  const int64_t groups = n + 1 < M ? n + 1 : M;  // non-empty groups, rows without an adapter among them
  L.max_tiles = M / kTileRows + groups;
  L.row = 4;
  L.perm = L.row + up4(M);
  L.off = L.perm + up4(M);
  L.tile = L.off + up4(n + 1);
  L.slot = L.tile + 4 * L.max_tiles;
  L.tile_ad = L.slot + up4(M);
  L.words = L.tile_ad + kMultiSlots * ((M + 127) / 128);  // tile rows are 128 rows or more
  return L;
}

// One CTA.  Rows are counted with shared-memory atomics (integer counts: any
// order gives the same), the counts scanned, and the rows placed warp by warp
// so that equal adapters keep the row order.
__global__ void __launch_bounds__(kPlanThreads)
    k_multi_plan(const int32_t* row_adapter, int M, int n, int32_t* plan,
                 int64_t o_row, int64_t o_perm, int64_t o_off, int64_t o_tile, int64_t o_slot,
                 int64_t o_tile_ad, int tile_rows) {
  pdl_wait();
  pdl_launch_dependents();
  // position counters of the adapters and, at [n], of the rows without one
  __shared__ int pos[WS_MULTI_MAX_ADAPTERS + 1];
  __shared__ int wsum[2][32];
  __shared__ int most_slots, too_many;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i <= n; i += kPlanThreads) pos[i] = 0;
  if (tid == 0) most_slots = too_many = 0;
  __syncthreads();
  for (int i = tid; i < M; i += kPlanThreads) {
    const int a = row_adapter[i];
    const bool has = a >= 0 && a < n;
    plan[o_row + i] = has ? a : -1;
    atomicAdd(&pos[has ? a : n], 1);
  }
  __syncthreads();
  // exclusive scan of rows and tiles over the n + 1 groups, kPer per thread
  constexpr int kPer = (WS_MULTI_MAX_ADAPTERS + 1 + kPlanThreads - 1) / kPlanThreads;
  int c[kPer], rows = 0, tiles = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = tid * kPer + k;
    c[k] = i <= n ? pos[i] : 0;
    rows += c[k];
    tiles += (c[k] + kTileRows - 1) / kTileRows;
  }
  int ir = rows, it = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int r = __shfl_up_sync(0xffffffffu, ir, o), t = __shfl_up_sync(0xffffffffu, it, o);
    if (lane >= o) ir += r, it += t;
  }
  if (lane == 31) wsum[0][warp] = ir, wsum[1][warp] = it;
  __syncthreads();
  int br = 0, bt = 0, all = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) br += wsum[0][w], bt += wsum[1][w];
    all += wsum[1][w];
  }
  if (tid == 0) plan[0] = all;
  int r0 = br + ir - rows, t0 = bt + it - tiles;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = tid * kPer + k;
    if (i <= n) {
      plan[o_off + i] = r0;
      pos[i] = r0;
      for (int q = 0; q < c[k]; q += kTileRows, ++t0)
        *reinterpret_cast<int4*>(plan + o_tile + 4 * (int64_t)t0) =
            make_int4(i < n ? i : -1, r0 + q, min(kTileRows, c[k] - q), 0);
      r0 += c[k];
    }
  }
  __syncthreads();
  for (int b = 0; b < M; b += kPlanThreads) {
    const int i = b + tid;
    int a = -1;
    if (i < M) {
      a = row_adapter[i];
      if (a < 0 || a >= n) a = n;
    }
    const uint32_t same = __match_any_sync(0xffffffffu, a);
    const int rank = __popc(same & ((1u << lane) - 1u));
    const int nw = min(kPlanThreads / 32, (M - b + 31) / 32);
    for (int w = 0; w < nw; ++w) {
      if (w == warp) {
        const int at = a >= 0 ? pos[a] + rank : 0;
        __syncwarp();
        if (a >= 0 && rank == 0) pos[a] += __popc(same);
        if (a >= 0) plan[o_perm + at] = i;
      }
      __syncthreads();
    }
  }
  // slots: one warp per tile row collects its adapters, 32 rows at a time
  for (int mt = warp; mt * (int64_t)tile_rows < M; mt += kPlanThreads / 32) {
    int32_t* list = plan + o_tile_ad + (int64_t)mt * kMultiSlots;
    int mine = -1, used = 0;  // lane l holds slot l's adapter
    const int end = min(M, (mt + 1) * tile_rows);
    for (int b = mt * tile_rows; b < end && used <= kMultiSlots; b += 32) {
      const int i = b + lane;
      int a = i < end ? row_adapter[i] : -1;
      if (a < 0 || a >= n) a = -1;
      int slot = -1;
      for (;;) {
        // lanes whose adapter has no slot yet
        for (int l = 0; l < used; ++l) {
          const int has = __shfl_sync(0xffffffffu, mine, l);
          if (a >= 0 && has == a) slot = l;
        }
        const uint32_t open = __ballot_sync(0xffffffffu, a >= 0 && slot < 0);
        if (!open) break;
        const int next = __shfl_sync(0xffffffffu, a, __ffs((int)open) - 1);
        if (used == kMultiSlots) {
          ++used;
          break;
        }
        if (lane == used) mine = next;
        ++used;
      }
      if (i < end) plan[o_slot + i] = slot;
    }
    if (lane < kMultiSlots) list[lane] = mine;
    if (lane == 0) {
      if (used > kMultiSlots) atomicOr(&too_many, 1);
      else atomicMax(&most_slots, used);
    }
  }
  __syncthreads();
  if (tid == 0) plan[1] = too_many ? -1 : most_slots;
}

// ------------------------------------------------------------------------ mma.sync pieces
// Two fp32 values as bf16 high parts and bf16 low parts (the remainders):
// together 16 significant bits or more.
WS_DEVINL void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x, y);
  lo = pack_bf16x2(x - bf16_lo(hi), y - bf16_hi(hi));
}
// Three parts: 24 bits, all of an fp32 value.
WS_DEVINL void split3(float x, float y, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_bf16x2(x, y);
  x -= bf16_lo(hi);
  y -= bf16_hi(hi);
  split2(x, y, mid, lo);
}
// Zeroes the halves of a bf16 pair whose keep bit (bits 0, 1 of b) is clear.
WS_DEVINL uint32_t keep2(uint32_t v, uint32_t b) {
  return v & (((b & 1u) ? 0x0000ffffu : 0u) | ((b & 2u) ? 0xffff0000u : 0u));
}

// ------------------------------------------------------------------------ skinny products
// out[row][0..16) = sum_c X~[row][c] F_a[.][c] for the rows of one tile (one
// adapter): U = (mask . x) A_a^T with F = A [16, C], or G = dY B_a with F = B
// [C, 16] (F_CJ).  X is bf16 and exact; an fp32 F enters as three bf16 parts,
// all of its bits (two parts cost U a factor of ten in error).
//
// Bound by reading X and the adapters once.  A cluster of CTAs shares a tile's
// contraction: its warps take the 64-deep steps in turn (a single-row tile of
// a decode batch then reads its adapter with 64 warps), the warps' sums are
// added in warp order, the CTAs' in rank order through distributed shared
// memory.  A lane reads 16 consecutive elements of a row (whole 128-byte
// lines per four lanes).
constexpr int kSkWarps = 8;
template <int V>
struct Int {
  static constexpr int value = V;
};
template <bool F_CJ, bool F16, bool MASKED>
__global__ void __launch_bounds__(kSkWarps * 32)
    k_multi_skinny(const uint16_t* X, const void* Fv, int64_t strideF,
                   int C, const uint32_t* mask, const int32_t* plan,
                   int64_t o_perm, int64_t o_tile, int64_t o_slot, float* out,
                   uint32_t* ext, int64_t M, uint32_t* zero) {
  __shared__ float part[kSkWarps][kTileRows * kR];
  __shared__ float sum[kTileRows * kR];
  const int lane = (int)lane_id(), warp = (int)warp_id(), g = lane >> 2, t = lane & 3;
  const int CS = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  pdl_wait();
  pdl_launch_dependents();
  // words the kernel that follows wants zeroed
  if (blockIdx.x == 0 && blockIdx.y == 0 && (int)threadIdx.x < kFewUnits) zero[threadIdx.x] = 0u;
  const int4 tile = *reinterpret_cast<const int4*>(plan + o_tile + 4 * (int64_t)blockIdx.y);  // (the table has room for it)
  if ((int)blockIdx.y >= plan[0]) return;  // the whole cluster alike
  const int32_t* rows = plan + o_perm + tile.y;
  const int cnt = tile.z, nsub = (cnt + 15) / 16;
  const int slots = ext ? plan[1] : 0;
  // a pair of results (r, j), (r, j + 1), i = r * 16 + j: fp32, and split into
  // bf16 parts [hi | lo | hi | lo] in the row's slot, zeros in the others: all
  // four products with [F_hi | F_hi | F_lo | F_lo] in one 64-deep step.  Two
  // parts hold 2^-17 of a value or better, so the term is off by 2^-16 at most
  // (root mean square 3.5e-6); six products of three parts would take a second
  // step for every slot.
  auto put = [&](int i, float v0, float v1) {
    const int64_t row = rows[i / kR];
    const int j = i % kR;
    *reinterpret_cast<float2*>(out + row * kR + j) = make_float2(v0, v1);
    if (slots <= 0) return;
    const int own = plan[o_slot + row];
    uint32_t hi, lo;
    split2(v0, v1, hi, lo);
    for (int l = 0; l < slots; ++l) {
      uint32_t* e = ext + ((int64_t)l * M + row) * 32 + j / 2;
      e[0] = l == own ? hi : 0u;
      e[8] = l == own ? lo : 0u;
      e[16] = l == own ? hi : 0u;
      e[24] = l == own ? lo : 0u;
    }
  };
  if (tile.x < 0) {  // rows without an adapter
    if (rank == 0)
      for (int i = 2 * threadIdx.x; i < cnt * kR; i += 2 * kSkWarps * 32) put(i, 0.0f, 0.0f);
    return;
  }
  float acc[4][2][4] = {};
  // one 64-deep step: the factor's fragments, then the rows 16 at a time.  The
  // step's products are summed by themselves and added in fp32: the tensor
  // cores cut off what a long running sum cannot hold.
  auto run = [&](auto ns) {
    constexpr int NS = decltype(ns)::value;
    int64_t ro[NS][2];  // row offsets (or -1) of this lane's rows of each 16-row part
#pragma unroll
    for (int u = 0; u < NS; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = u * 16 + h * 8 + g;
        ro[u][h] = r < cnt ? (int64_t)rows[r] * C : -1;
      }
    struct Fac {
      uint4 w[F16 ? 4 : 8];  // this lane's 16 values for j = g and for j = g + 8
    };
    auto load_f = [&](Fac& f, int st) {
      const int c0 = st * 64 + 16 * t;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int j = nt * 8 + g;
        if constexpr (F16) {
          const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(Fv) + tile.x * strideF + (int64_t)j * C + c0);
          f.w[2 * nt] = p[0], f.w[2 * nt + 1] = p[1];
        } else if constexpr (F_CJ) {
          const uint32_t* p = static_cast<const uint32_t*>(Fv) + tile.x * strideF + (int64_t)c0 * kR + j;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            f.w[4 * nt + q] = make_uint4(p[(4 * q) * kR], p[(4 * q + 1) * kR], p[(4 * q + 2) * kR], p[(4 * q + 3) * kR]);
        } else {
          const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(Fv) + tile.x * strideF + (int64_t)j * C + c0);
#pragma unroll
          for (int q = 0; q < 4; ++q) f.w[4 * nt + q] = p[q];
        }
      }
    };
    struct Row {
      uint4 x[2][2];
      uint32_t keep[2];
    };
    auto load_x = [&](Row& r, int st, int u) {
      const int c0 = st * 64 + 16 * t;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        r.x[h][0] = r.x[h][1] = make_uint4(0u, 0u, 0u, 0u);
        r.keep[h] = 0xffffu;
        if (ro[u][h] >= 0) {
          const uint4* p = reinterpret_cast<const uint4*>(X + ro[u][h] + c0);
          r.x[h][0] = p[0], r.x[h][1] = p[1];
          if constexpr (MASKED) r.keep[h] = mask[(ro[u][h] + c0) >> 5] >> (c0 & 31);
        }
      }
    };
    const int step = kSkWarps * CS;
    int st = rank * kSkWarps + warp;
    const int end = C / 64;
    // Ahead of the registers, which hold one step of the factor and 16 rows: the
    // lines of two steps ahead are asked for, and of tiles of more than 16 rows
    // those rows', a lane for its two (333 rows of 27648: 21 us; 23 without the
    // factor's, 26 with neither; two 16-row parts in registers gave no more).
    int64_t po[2] = {-1, -1};
    auto ask = [&](int s) {
      // the factor's lines: 32 in fp32 (two for each of 16 rows, or all of [64, 16]), 16 in bf16
      const int64_t at = F_CJ ? (int64_t)s * 64 * kR + lane * 32
                              : (F16 ? (int64_t)(lane & 15) * C + s * 64 : (int64_t)(lane >> 1) * C + s * 64 + (lane & 1) * 32);
      asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t*>(Fv) + (tile.x * strideF + at) * (F16 ? 2 : 4)));
#pragma unroll
      for (int h = 0; h < NS / 2; ++h)
        if (po[h] >= 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(X + po[h] + s * 64));
    };
    Fac f;
    Row r;
    if (st < end) {
      load_f(f, st);
      load_x(r, st, 0);
#pragma unroll
      for (int h = 0; h < NS / 2; ++h)
        if (h * 32 + lane < cnt) po[h] = (int64_t)rows[h * 32 + lane] * C;
      ask(st);
      if (st + step < end) ask(st + step);
    }
    for (; st < end; st += step) {
      uint32_t b[F16 ? 1 : 3][2][4][2];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          if constexpr (F16) {
            const uint4 q = f.w[2 * nt + s / 2];
            b[0][nt][s][0] = (s & 1) ? q.z : q.x;
            b[0][nt][s][1] = (s & 1) ? q.w : q.y;
          } else {
            const uint4 q = f.w[4 * nt + s];
            split3(__uint_as_float(q.x), __uint_as_float(q.y), b[0][nt][s][0], b[1][nt][s][0], b[2][nt][s][0]);
            split3(__uint_as_float(q.z), __uint_as_float(q.w), b[0][nt][s][1], b[1][nt][s][1], b[2][nt][s][1]);
          }
        }
      const bool more = st + step < end;
      if (more) load_f(f, st + step);
      if (st + 2 * step < end) ask(st + 2 * step);
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        uint32_t x[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[h][0] = r.x[h][0].x, x[h][1] = r.x[h][0].y, x[h][2] = r.x[h][0].z, x[h][3] = r.x[h][0].w;
          x[h][4] = r.x[h][1].x, x[h][5] = r.x[h][1].y, x[h][6] = r.x[h][1].z, x[h][7] = r.x[h][1].w;
          if constexpr (MASKED) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[h][e] = keep2(x[h][e], r.keep[h] >> (2 * e));
          }
        }
        if (u + 1 < NS) load_x(r, st, u + 1);
        else if (more) load_x(r, st + step, 0);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          float d[4] = {};
#pragma unroll
          for (int k = F16 ? 0 : 2; k >= 0; --k)  // small parts first
#pragma unroll
            for (int s = 0; s < 4; ++s)
              mma16816(d, x[0][2 * s], x[1][2 * s], x[0][2 * s + 1], x[1][2 * s + 1], b[k][nt][s][0], b[k][nt][s][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[u][nt][e] += d[e];
        }
      }
    }
  };
  if (nsub == 1) run(Int<1>{});
  else if (nsub == 2) run(Int<2>{});
  else run(Int<4>{});
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (u >= nsub) break;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(&part[warp][(u * 16 + h * 8 + g) * kR + nt * 8 + 2 * t]) =
            make_float2(acc[u][nt][2 * h], acc[u][nt][2 * h + 1]);
  }
  __syncthreads();
  const int elems = cnt * kR;
  for (int i = 2 * threadIdx.x; i < elems; i += 2 * kSkWarps * 32) {
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kSkWarps; ++w) {
      const float2 p = *reinterpret_cast<const float2*>(&part[w][i]);
      s.x += p.x;
      s.y += p.y;
    }
    if (CS == 1) put(i, s.x, s.y);
    else *reinterpret_cast<float2*>(&sum[i]) = s;
  }
  if (CS == 1) return;
  cluster_sync();
  for (int i = 2 * (rank * kSkWarps * 32 + threadIdx.x); i < elems; i += 2 * CS * kSkWarps * 32) {
    float2 s = make_float2(0.0f, 0.0f);
    for (int c = 0; c < CS; ++c) {
      float x, y;
      asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                   : "=f"(x), "=f"(y)
                   : "r"(mapa_shared(smem_u32(&sum[i]), (uint32_t)c))
                   : "memory");
      s.x += x;
      s.y += y;
    }
    put(i, s.x, s.y);
  }
  cluster_sync();  // the sums stay until every CTA of the cluster has read them
}

// ------------------------------------------------------------------------ weight gradients
// One launch for both gradients of every adapter:
//   dB_a [N, 16] = s_a sum_{m of a} dY[m]^T U[m],  dA_a [16, K] = s_a sum_{m of a} G[m]^T (mask . x)[m]
// CTA = 128 columns of dY or x for one adapter: four warps take the adapter's
// rows in turn, 16 at a time, for each 64 columns, D (16 x 64) += P^T Q, and
// their sums are added in warp order.  Q is bf16 and exact, the fp32 P enters
// as three bf16 parts.  A lane takes 8 consecutive columns of four rows and
// pairs rows with byte permutes: column 8g + i of the tile is column g of the
// i-th 8-wide product, so nothing is transposed.  Bound by reading dY and x
// once; each warp keeps kWgStages steps of rows on their way through a ring of
// its own in shared memory (with one step ahead in registers the pass over
// 2048 rows of 5120 + 27648 columns took 70 us, this way 55: 2.4 TB/s of the
// 134 MB; ALU 42%, the byte permutes and splits, at two CTAs an SM).
constexpr int kWgWarps = 8, kWgSplit = 4, kWgStages = 4;
constexpr int kWgQ = 16 * 128, kWgP = 16 * 80, kWgM = 16 * 8;  // bytes of a step: Q, P (rows padded), mask
constexpr int kWgStage = kWgQ + kWgP + kWgM;
constexpr int kWgSmem = kWgWarps * kWgStages * kWgStage;
static_assert(kWgSmem >= kWgWarps * kR * 64 * 4, "the sums fit the ring");
struct WgArgs {
  const float* P[2];      // U, G  [M, 16]
  const uint16_t* Q[2];   // dY [M, C0], x [M, C1]
  float* out[2];          // dB, dA
  int C[2];
  int64_t stride[2];
  const uint32_t* mask;   // of Q[1], or NULL
  const float* scale;
  const int32_t* plan;
  int64_t o_perm, o_off;
  int accumulate;
};
WS_DEVINL uint32_t lo_pair(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
WS_DEVINL uint32_t hi_pair(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

__global__ void __launch_bounds__(kWgWarps * 32, 2) k_multi_wgrad(const WgArgs w) {
  extern __shared__ __align__(128) uint8_t wg_smem[];
  float(*red)[kR][64] = reinterpret_cast<float(*)[kR][64]>(wg_smem);
  const int lane = (int)lane_id(), warp = (int)warp_id(), g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_launch_dependents();
  const int a = blockIdx.y;
  const int r_beg = w.plan[w.o_off + a], cnt = w.plan[w.o_off + a + 1] - r_beg;
  if (cnt == 0 && w.accumulate) return;
  const int nb = (w.C[0] + 127) / 128;
  const int which = (int)blockIdx.x >= nb ? 1 : 0;
  const int C = which ? w.C[1] : w.C[0];
  const int cta0 = ((int)blockIdx.x - (which ? nb : 0)) * 128;
  const int col0 = cta0 + (warp / kWgSplit) * 64, part = warp % kWgSplit;
  const bool cols = col0 < C;
  const float* P = which ? w.P[1] : w.P[0];
  const uint16_t* Q = (which ? w.Q[1] : w.Q[0]) + col0;
  const uint32_t* mask = which ? w.mask : nullptr;
  const int32_t* rows = w.plan + w.o_perm + r_beg;
  float d[8][4] = {};
  if (cols) {
    uint8_t* ring = wg_smem + warp * kWgStages * kWgStage;
    constexpr int kHop = kWgSplit * 16;
    // lane l < 16 holds the row of place l of the step that is fetched next
    int s_idx = part * 16;
    auto next_idx = [&]() {
      const int r = s_idx + (lane & 15);
      s_idx += kHop;
      return r < cnt ? rows[r] : -1;
    };
    int idx = next_idx();
    int slot_in = 0;
    // 16-byte chunk c of row r of Q at chunk place c ^ (r & 7); rows past the
    // end arrive as zeros
    auto fetch = [&]() {
      const uint32_t base = smem_u32(ring + slot_in * kWgStage);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 4 + lane / 8, c = lane % 8;
        const int64_t row = __shfl_sync(0xffffffffu, idx, r);
        cp_async16(base + (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)), Q + (row < 0 ? 0 : row * C + c * 8), row < 0 ? 0u : 16u);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = i * 8 + lane / 4, c = lane % 4;
        const int64_t row = __shfl_sync(0xffffffffu, idx, r);
        cp_async16(base + (uint32_t)(kWgQ + r * 80 + c * 16), P + (row < 0 ? 0 : row * kR + c * 4), row < 0 ? 0u : 16u);
      }
      if (mask) {
        const int64_t row = __shfl_sync(0xffffffffu, idx, lane / 2);
        cp_async4(base + (uint32_t)(kWgQ + kWgP + lane * 4), mask + (row < 0 ? 0 : (row * C + col0) / 32 + (lane & 1)), row < 0 ? 0u : 4u);
      }
      cp_async_commit();
      if (++slot_in == kWgStages) slot_in = 0;
      idx = next_idx();
    };
#pragma unroll
    for (int i = 0; i < kWgStages - 1; ++i) fetch();
    int slot = 0;
    for (int s0 = part * 16; s0 < cnt; s0 += kHop) {
      cp_async_wait<kWgStages - 2>();
      __syncwarp();  // the step is there for every lane, and the slot before it is free
      const uint8_t* st = ring + slot * kWgStage;
      uint32_t q[4][4];
      float p[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // rows 2t, 2t+1, 2t+8, 2t+9
        const int r = 2 * t + (i & 1) + (i >> 1) * 8;
        const uint4 v = *reinterpret_cast<const uint4*>(st + r * 128 + ((g ^ (r & 7)) << 4));
        q[i][0] = v.x, q[i][1] = v.y, q[i][2] = v.z, q[i][3] = v.w;
        p[i][0] = *reinterpret_cast<const float*>(st + kWgQ + r * 80 + g * 4);
        p[i][1] = *reinterpret_cast<const float*>(st + kWgQ + r * 80 + g * 4 + 32);
        if (mask) {
          const uint32_t keep = *reinterpret_cast<const uint32_t*>(st + kWgQ + kWgP + r * 8 + (g / 4) * 4) >> (8 * (g & 3));
#pragma unroll
          for (int k = 0; k < 4; ++k) q[i][k] = keep2(q[i][k], keep >> (2 * k));
        }
      }
      __syncwarp();
      fetch();
      if (++slot == kWgStages) slot = 0;
      uint32_t ah[4], am[4], al[4];
      split3(p[0][0], p[1][0], ah[0], am[0], al[0]);
      split3(p[0][1], p[1][1], ah[1], am[1], al[1]);
      split3(p[2][0], p[3][0], ah[2], am[2], al[2]);
      split3(p[2][1], p[3][1], ah[3], am[3], al[3]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = i / 2;
        const uint32_t b0 = (i & 1) ? hi_pair(q[0][k], q[1][k]) : lo_pair(q[0][k], q[1][k]);
        const uint32_t b1 = (i & 1) ? hi_pair(q[2][k], q[3][k]) : lo_pair(q[2][k], q[3][k]);
        // The step by itself, small parts first, then one fp32 addition that
        // rounds: the tensor cores cut off what a long running sum cannot hold
        // (one adapter of 262144 rows of one sign: 4.4e-4 off that way, always
        // towards zero; at most 1.7e-6 this way, 2 us of 545 more at 2048 rows).
        float e[4] = {};
        mma16816(e, al[0], al[1], al[2], al[3], b0, b1);
        mma16816(e, am[0], am[1], am[2], am[3], b0, b1);
        mma16816(e, ah[0], ah[1], ah[2], ah[3], b0, b1);
#pragma unroll
        for (int z = 0; z < 4; ++z) d[i][z] += e[z];
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();  // the ring becomes the sums
  const int nw = min(kWgSplit, (cnt + 15) / 16);  // parts that had rows
  if (part < nw) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 8; i += 4)
          *reinterpret_cast<float4*>(&red[warp][g + 8 * h][(2 * t + c) * 8 + i]) =
              make_float4(d[i][2 * h + c], d[i + 1][2 * h + c], d[i + 2][2 * h + c], d[i + 3][2 * h + c]);
  }
  __syncthreads();
  const float s = cnt > 0 ? w.scale[a] : 0.0f;  // (no rows: zeros, whatever the scale)
  float* out = (which ? w.out[1] : w.out[0]) + a * (which ? w.stride[1] : w.stride[0]);
  // four results a thread at a time: along k for dA [16, K], along j for dB [N, 16]
#pragma unroll
  for (int k = 0; k < 2 * kR * 64 / (kWgWarps * 32 * 4); ++k) {
    const int i = (k * kWgWarps * 32 + (int)threadIdx.x) * 4;
    const int grp = i / (kR * 64), e = i % (kR * 64);
    const int j = which ? e / 64 : e % kR, c = which ? e % 64 : e / kR;
    if (cta0 + grp * 64 >= C) continue;
    float v[4] = {};
    for (int x = 0; x < nw; ++x)
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] += which ? red[grp * kWgSplit + x][j][c + u] : red[grp * kWgSplit + x][j + u][c];
    float4* o = reinterpret_cast<float4*>(out + (which ? (int64_t)j * C + cta0 + grp * 64 + c
                                                       : (int64_t)(cta0 + grp * 64 + c) * kR + j));
    // rounded by themselves: accumulating adds the finished contribution once
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = __fmul_rn(v[u], s);
    if (w.accumulate) {
      const float4 old = *o;
      v[0] = old.x + v[0], v[1] = old.y + v[1], v[2] = old.z + v[2], v[3] = old.w + v[3];
    }
    *o = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// ------------------------------------------------------------------------ the adapter term by itself
// Where a tile row of the GEMM has more adapters than slots (many requests of
// few rows): out = base + the adapter term, one rounding.  FWD: + s_a sum_j
// U[m][j] B_a[n][j]; else + mask . s_a sum_j G[m][j] A_a[j][k].  CTA = 16 rows
// of one tile of the plan (one adapter) x 256 columns; a thread keeps the factor
// of its two columns in registers for all rows and has eight rows of the base on
// their way at a time; bound by the fp32 base it reads and what it writes.  A
// slot costs the GEMM a 64-deep step of every tile: 512 rows of 5120x5120 take
// 57 us with 8 adapters in slots, 73 with 16, 324 with the term in the GEMM's
// epilogue, 62 this way (64 adapters).
constexpr int kExThreads = 128, kExRows = 16;
template <bool FWD, bool F16, bool O16>
__global__ void __launch_bounds__(kExThreads)
    k_multi_expand(const float* base, const float* P, const void* Fv, int64_t strideF, const float* scale,
                   const uint32_t* mask, const int32_t* plan, int64_t o_perm, int64_t o_tile, int C, int accumulate,
                   void* out) {
  __shared__ float u[kExRows][kR];
  __shared__ int rows[kExRows];
  pdl_wait();
  pdl_launch_dependents();
  const int4 tile = *reinterpret_cast<const int4*>(plan + o_tile + 4 * (int64_t)blockIdx.y);  // (the table has room for it)
  if (plan[1] >= 0 || (int)blockIdx.y >= plan[0]) return;
  const int a = tile.x, r0 = (int)blockIdx.z * kExRows, cnt = min(kExRows, tile.z - r0);
  if (cnt <= 0) return;
  const float s = a >= 0 ? scale[a] : 0.0f;
  for (int i = threadIdx.x; i < cnt * kR; i += kExThreads) {
    const int row = plan[o_perm + tile.y + r0 + i / kR];
    if (i % kR == 0) rows[i / kR] = row;
    u[i / kR][i % kR] = a >= 0 ? s * P[(int64_t)row * kR + i % kR] : 0.0f;
  }
  __syncthreads();
  const int c = ((int)blockIdx.x * kExThreads + (int)threadIdx.x) * 2;
  if (c >= C) return;
  float f0[kR], f1[kR];  // the factor of columns c and c + 1
#pragma unroll
  for (int j = 0; j < kR; ++j) f0[j] = f1[j] = 0.0f;
  if (a >= 0) {
    if constexpr (!FWD) {
      const float* F = static_cast<const float*>(Fv) + a * strideF + c;
#pragma unroll
      for (int j = 0; j < kR; ++j) {
        const float2 v = *reinterpret_cast<const float2*>(F + (int64_t)j * C);
        f0[j] = v.x, f1[j] = v.y;
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float* f = h ? f1 : f0;
        const int64_t o = a * strideF + (int64_t)(c + h) * kR;
#pragma unroll
        for (int j = 0; j < kR; j += 4) {
          if constexpr (F16) {
            const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(Fv) + o + j);
            f[j] = bf16_lo(v.x), f[j + 1] = bf16_hi(v.x), f[j + 2] = bf16_lo(v.y), f[j + 3] = bf16_hi(v.y);
          } else {
            const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(Fv) + o + j);
            f[j] = v.x, f[j + 1] = v.y, f[j + 2] = v.z, f[j + 3] = v.w;
          }
        }
      }
    }
  }
  for (int rb = 0; rb < cnt; rb += 8) {
    float2 base8[8];
    uint32_t keep[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t at = (int64_t)rows[min(rb + i, cnt - 1)] * C + c;
      base8[i] = *reinterpret_cast<const float2*>(base + at);
      keep[i] = !FWD && mask ? mask[at >> 5] >> (at & 31) : 3u;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = rb + i;
      if (r >= cnt) break;
      const int64_t at = (int64_t)rows[r] * C + c;
      float2 v = base8[i];
      float d0 = 0.0f, d1 = 0.0f;
#pragma unroll
      for (int j = 0; j < kR; j += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&u[r][j]);
        d0 = fmaf(x.x, f0[j], d0), d0 = fmaf(x.y, f0[j + 1], d0), d0 = fmaf(x.z, f0[j + 2], d0), d0 = fmaf(x.w, f0[j + 3], d0);
        d1 = fmaf(x.x, f1[j], d1), d1 = fmaf(x.y, f1[j + 1], d1), d1 = fmaf(x.z, f1[j + 2], d1), d1 = fmaf(x.w, f1[j + 3], d1);
      }
      if (a >= 0) {
        if (keep[i] & 1u) v.x += d0;
        if (keep[i] & 2u) v.y += d1;
      }
      if constexpr (O16) {
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + at) = pack_bf16x2(v.x, v.y);
      } else {
        float2* o = reinterpret_cast<float2*>(static_cast<float*>(out) + at);
        if (accumulate) {
          const float2 old = *o;
          v.x = old.x + v.x, v.y = old.y + v.y;
        }
        *o = v;
      }
    }
  }
}

// ------------------------------------------------------------------------ host side
#ifndef WS_FEW_ROWS
#define WS_FEW_ROWS 64
#endif
constexpr int kFewRows = WS_FEW_ROWS;  // rows up to which run_few makes the forward
// Whether run_few_bwd makes the input gradient, and not the tensor-core GEMM: up
// to 32 rows always (backward of 32 rows, weights from DRAM, in a graph: 16.0 us
// against 21.5 at 896 x 896, 76 against 109 at 27648 x 5120), up to 64 with eight
// steps of 128 x 256 weights for every SM (64 rows: 5120 x 5120, 5.3 steps, 42.6
// against 42.6; 3584 x 18944, 13.6 steps, 59 against 64; 27648 x 5120, 28 steps, 92
// against 114; 896 x 896 27.6 against 23.0).
bool few_makes_dx(int64_t M, int64_t N, int64_t K) {
  return M <= 32 || (M <= kFewRows && (K + 127) / 128 * ((N + 255) / 256) >= 8 * device_sm_count());
}

struct WsLayout {
  size_t G, ext, words, base, partial, total;
};
// words: kFewUnits words that the skinny product zeroes for the kernel after it.
// run_few: a flag for each CTA; the GEMM: the word of bad values, then the flags
// (from the caller's workspace, and not the library's ring: a captured graph
// keeps the words it was given, and the ring comes round to them again).
// base: the fp32 base term of k_multi_expand, which a set of no more adapters
// than slots never needs.
WsLayout ws_layout(int64_t M, int64_t N, int64_t K, int32_t n) {
  WsLayout L{};
  const size_t pf = gemm_multi_bytes(plan_gemm(false, M, N, K), M, N), pb = gemm_multi_bytes(plan_gemm(true, M, K, N), M, K);
  L.G = 0;
  L.ext = al256((size_t)M * kR * 4);
  L.words = L.ext + (size_t)M * kMultiSlots * 128;
  L.base = L.words + kFewUnits * 4;
  L.partial = L.base + (n > kMultiSlots ? al256((size_t)M * (size_t)(N > K ? N : K) * 4) : 0);
  size_t p = pf > pb ? pf : pb;
  if (M <= kFewRows && p < kFewUnits * 64 * 128 * 4) p = kFewUnits * 64 * 128 * 4;
  L.total = L.partial + al256(p);
  return L;
}

template <typename K, typename... Args>
cudaError_t launch_cluster(K k, dim3 grid, int threads, int cluster, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// CTAs that share a tile's contraction: as many as have a step for every warp
// and fit the GPU at once (two an SM) with the most tiles a batch can have.
int skinny_cluster(int64_t C, int64_t tiles) {
  int cs = 8;
  while (cs > 1 && (cs * kSkWarps > C / 64 || cs * tiles > 2 * device_sm_count())) cs /= 2;
  return cs;
}

cudaError_t run_skinny(bool f_cj, const uint16_t* X, const void* F, bool f16, int64_t strideF, int64_t C,
                       const uint32_t* mask, const ws_lora_plan& plan, float* out, uint8_t* ws,
                       const WsLayout& W, bool slots, cudaStream_t st) {
  const PlanLayout L = plan_layout(plan.M, plan.n_adapters);
  const int cs = skinny_cluster(C, L.max_tiles);
  auto k = f_cj ? k_multi_skinny<true, false, false>
                : (f16 ? (mask ? k_multi_skinny<false, true, true> : k_multi_skinny<false, true, false>)
                       : (mask ? k_multi_skinny<false, false, true> : k_multi_skinny<false, false, false>));
  return launch_cluster(k, dim3((unsigned)cs, (unsigned)L.max_tiles), kSkWarps * 32, cs, 0, st, X, F, strideF,
                        (int)C, mask, (const int32_t*)plan.data, L.perm, L.tile, L.slot, out,
                        slots ? reinterpret_cast<uint32_t*>(ws + W.ext) : nullptr, plan.M,
                        reinterpret_cast<uint32_t*>(ws + W.words));
}
static_assert(kFewUnits <= kSkWarps * 32, "one thread zeroes each word");

// The GEMM's view of the adapter term with P = U or G and F = B or A.
MultiLora multi_of(const ws_lora_plan& plan, uint8_t* ws, const WsLayout& W, const float* P, const void* F, bool f16,
                   int64_t stride, const float* scale) {
  const PlanLayout L = plan_layout(plan.M, plan.n_adapters);
  const int32_t* pl = static_cast<const int32_t*>(plan.data);
  MultiLora m{};
  m.P = P;
  m.ext = reinterpret_cast<const uint16_t*>(ws + W.ext);
  m.F = F;
  m.scale = scale;
  m.row = pl + L.row;
  m.slots = pl + 1;
  m.tile_ad = pl + L.tile_ad;
  m.bad = reinterpret_cast<uint32_t*>(ws + W.words);
  m.flags = m.bad + 1;
  m.out32 = reinterpret_cast<float*>(ws + W.base);
  m.stride = stride;
  m.f16 = f16 ? 1 : 0;
  return m;
}

template <typename K>
cudaError_t run_expand(K k, const MultiLora& ml, const uint32_t* mask, const ws_lora_plan& plan, int64_t C,
                       int accumulate, void* out, cudaStream_t st) {
  const PlanLayout L = plan_layout(plan.M, plan.n_adapters);
  note_launch();
  return launch_pdl(k, dim3((unsigned)((C + 2 * kExThreads - 1) / (2 * kExThreads)), (unsigned)L.max_tiles,
                             kTileRows / kExRows),
                    dim3(kExThreads), 0, st, (const float*)ml.out32, ml.P, ml.F, ml.stride, ml.scale, mask,
                    (const int32_t*)plan.data, L.perm, L.tile, (int)C, accumulate, out);
}

FewArgs few_args(const ws_nf4* W, const uint16_t* x, const ws_lora_plan& plan, const float* P, const void* F,
                 int64_t stride, const float* scale, void* y, uint8_t* ws, const WsLayout& L) {
  FewArgs a{};
  a.codes = W->codes, a.absmax = W->absmax, a.x = x;
  a.M = (int)plan.M, a.N = (int)W->N, a.K = (int)W->K;
  a.P = P, a.F = F, a.stride = stride, a.scale = scale;
  a.row = static_cast<const int32_t*>(plan.data) + plan_layout(plan.M, plan.n_adapters).row;
  a.y = y;
  a.partial = reinterpret_cast<float*>(ws + L.partial);
  a.flags = reinterpret_cast<uint32_t*>(ws + L.words);
  return a;
}

ws_status check_plan(const ws_lora_plan* p) {
  if (!p || !p->data) return WS_ERR_INVALID;
  if (p->M < 1 || p->M > (1 << 20) || p->n_adapters < 1 || p->n_adapters > WS_MULTI_MAX_ADAPTERS) return WS_ERR_SHAPE;
  if (!al16p(p->data)) return WS_ERR_ALIGN;
  return WS_OK;
}

// The shapes that the calls take (and their workspace is sized for).
bool shape_ok(int64_t M, int64_t N, int64_t K, int32_t n) {
  return M >= 1 && M <= (1 << 20) && n >= 1 && n <= WS_MULTI_MAX_ADAPTERS && N >= 64 && K >= 64 && N % 64 == 0 &&
         K % 64 == 0 && N <= (1 << 30) && K <= (1 << 30) && (double)M * (double)(N > K ? N : K) < 17179869184.0;  // 2^34
}

// What forward and backward check alike.
ws_status check_multi(const ws_nf4* W, const ws_lora_set* set, const ws_lora_plan* plan,
                      const uint32_t* mask) {
  const ws_status s = check_plan(plan);
  if (s != WS_OK) return s;
  if (!W || !W->codes || !W->absmax || !set || !set->A || !set->B || !set->scale) return WS_ERR_INVALID;
  if (set->dtype != WS_DTYPE_F32 && set->dtype != WS_DTYPE_BF16) return WS_ERR_INVALID;
  if (!shape_ok(plan->M, W->N, W->K, plan->n_adapters)) return WS_ERR_SHAPE;
  if (set->r != kR || set->n_adapters != plan->n_adapters) return WS_ERR_SHAPE;
  if (set->stride_a < kR * W->K || set->stride_b < kR * W->N || set->stride_a % 8 || set->stride_b % 8) return WS_ERR_SHAPE;
  if (!al16p(W->codes) || !al16p(W->absmax) || !al16p(set->A) || !al16p(set->B) || !al16p(mask)) return WS_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(set->scale) & 3u) return WS_ERR_ALIGN;
  return WS_OK;
}

NF4View view(const ws_nf4* W) {
  NF4View v;
  v.codes = W->codes;
  v.absmax = W->absmax;
  v.N = W->N;
  v.K = W->K;
  return v;
}

#define WS_RUN(x)                                \
  do {                                           \
    if ((x) != cudaSuccess) return WS_ERR_CUDA;  \
  } while (0)

}  // namespace

}  // namespace ws

using namespace ws;

extern "C" {

ws_status ws_dropout_mask(ws_dropout_key key, int64_t M, int64_t K, uint32_t* mask, ws_stream_t stream) {
  if (!mask) return WS_ERR_INVALID;
  if (M < 1 || K < 64 || K % 64 || (double)M * (double)K >= 17179869184.0) return WS_ERR_SHAPE;
  if (!(key.p >= 0.0 && key.p < 1.0) || key.linear > 255u || key.microbatch > 0xFFFFFFu) return WS_ERR_INVALID;
  if (!al16p(mask)) return WS_ERR_ALIGN;
  WS_RUN(run_mask_gen(M, K, make_drop_key(key), mask, (cudaStream_t)stream));
  return WS_OK;
}

ws_status ws_lora_multi_plan_size(int64_t M, int32_t n_adapters, size_t* bytes) {
  if (!bytes) return WS_ERR_INVALID;
  if (M < 1 || M > (1 << 20) || n_adapters < 1 || n_adapters > WS_MULTI_MAX_ADAPTERS) return WS_ERR_SHAPE;
  *bytes = (size_t)plan_layout(M, n_adapters).words * 4;
  return WS_OK;
}

ws_status ws_lora_multi_plan_init(const ws_lora_plan* plan, const int32_t* row_adapter,
                                  ws_stream_t stream) {
  const ws_status s = check_plan(plan);
  if (s != WS_OK) return s;
  if (!row_adapter) return WS_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(row_adapter) & 3u) return WS_ERR_ALIGN;
  const PlanLayout L = plan_layout(plan->M, plan->n_adapters);
  note_launch();
  WS_RUN(launch_pdl(k_multi_plan, dim3(1), dim3(kPlanThreads), 0, (cudaStream_t)stream, row_adapter,
                    (int)plan->M, (int)plan->n_adapters, (int32_t*)plan->data, L.row, L.perm, L.off, L.tile,
                    L.slot, L.tile_ad, (int)gemm_tile_rows(plan->M)));
  return WS_OK;
}

ws_status ws_lora_multi_workspace_size(int64_t M, int64_t N, int64_t K, int32_t n_adapters,
                                       size_t* bytes) {
  if (!bytes) return WS_ERR_INVALID;
  if (!shape_ok(M, N, K, n_adapters)) return WS_ERR_SHAPE;
  *bytes = ws_layout(M, N, K, n_adapters).total;
  return WS_OK;
}

ws_status ws_lora_linear_fwd_multi(const ws_nf4* W, const uint16_t* x, const ws_lora_set* set,
                                   const ws_lora_plan* plan, const uint32_t* mask, uint16_t* y,
                                   float* U_saved, void* workspace, size_t ws_bytes,
                                   ws_stream_t stream) {
  const ws_status s = check_multi(W, set, plan, mask);
  if (s != WS_OK) return s;
  if (!x || !y || !U_saved || !workspace) return WS_ERR_INVALID;
  if (!al16p(x) || !al16p(y) || !al16p(U_saved) || !al16p(workspace)) return WS_ERR_ALIGN;
  const int64_t M = plan->M, N = W->N, K = W->K;
  const WsLayout L = ws_layout(M, N, K, set->n_adapters);
  if (ws_bytes < L.total) return WS_ERR_OOM;
  cudaStream_t st = (cudaStream_t)stream;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool f16 = set->dtype == WS_DTYPE_BF16;
  if (M <= kFewRows) {
    const FewArgs a = few_args(W, x, *plan, U_saved, set->B, set->stride_b, set->scale, y, ws, L);
    WS_RUN(run_skinny(false, x, set->A, f16, set->stride_a, K, mask, *plan, U_saved, ws, L, false, st));
    WS_RUN(run_few(a, f16, st));
    return WS_OK;
  }
  WS_RUN(run_skinny(false, x, set->A, f16, set->stride_a, K, mask, *plan, U_saved, ws, L, true, st));
  const MultiLora ml = multi_of(*plan, ws, L, U_saved, set->B, f16, set->stride_b, set->scale);
  WS_RUN(run_nf4_gemm_multi(plan_gemm(false, M, N, K), view(W), x, M, ml, nullptr, y, 0, 0,
                            reinterpret_cast<float*>(ws + L.partial), st));
  if (set->n_adapters > kMultiSlots)
    WS_RUN(run_expand(f16 ? k_multi_expand<true, true, true> : k_multi_expand<true, false, true>, ml, nullptr, *plan,
                      N, 0, y, st));
  return WS_OK;
}

ws_status ws_lora_linear_bwd_multi(const ws_nf4* W, const uint16_t* x, const ws_lora_set* set,
                                   const ws_lora_plan* plan, const uint32_t* mask,
                                   const float* U_saved, const uint16_t* dY, void* dX,
                                   int32_t dX_dtype, int32_t accumulate, float* dA, float* dB,
                                   void* workspace, size_t ws_bytes, ws_stream_t stream) {
  const ws_status s = check_multi(W, set, plan, mask);
  if (s != WS_OK) return s;
  if (!x || !U_saved || !dY || !dX || !dA || !dB || !workspace) return WS_ERR_INVALID;
  if (dX_dtype != WS_DTYPE_BF16 && dX_dtype != WS_DTYPE_F32) return WS_ERR_INVALID;
  if (accumulate & ~(WS_ACC_DX | WS_ACC_GRADS)) return WS_ERR_INVALID;
  if ((accumulate & WS_ACC_DX) && dX_dtype != WS_DTYPE_F32) return WS_ERR_INVALID;
  if (set->dtype != WS_DTYPE_F32) return WS_ERR_UNSUPPORTED;
  if (!al16p(x) || !al16p(U_saved) || !al16p(dY) || !al16p(dX) || !al16p(dA) || !al16p(dB) || !al16p(workspace))
    return WS_ERR_ALIGN;
  const int64_t M = plan->M, N = W->N, K = W->K;
  const WsLayout L = ws_layout(M, N, K, set->n_adapters);
  if (ws_bytes < L.total) return WS_ERR_OOM;
  cudaStream_t st = (cudaStream_t)stream;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int32_t* pl = static_cast<const int32_t*>(plan->data);
  const PlanLayout P = plan_layout(M, plan->n_adapters);
  float* G = reinterpret_cast<float*>(ws + L.G);
  WS_RUN(run_skinny(true, dY, set->B, false, set->stride_b, N, nullptr, *plan, G, ws, L, !few_makes_dx(M, N, K), st));
  WgArgs w{};
  w.P[0] = U_saved, w.P[1] = G;
  w.Q[0] = dY, w.Q[1] = x;
  w.out[0] = dB, w.out[1] = dA;
  w.C[0] = (int)N, w.C[1] = (int)K;
  w.stride[0] = set->stride_b, w.stride[1] = set->stride_a;
  w.mask = mask;
  w.scale = set->scale;
  w.plan = pl;
  w.o_perm = P.perm, w.o_off = P.off;
  w.accumulate = (accumulate & WS_ACC_GRADS) ? 1 : 0;
  static const cudaError_t attr =
      cudaFuncSetAttribute(k_multi_wgrad, cudaFuncAttributeMaxDynamicSharedMemorySize, kWgSmem);
  WS_RUN(attr);
  note_launch();
  WS_RUN(launch_pdl(k_multi_wgrad, dim3((unsigned)((N + 127) / 128 + (K + 127) / 128), (unsigned)set->n_adapters), dim3(kWgWarps * 32),
                    kWgSmem, st, w));
  if (few_makes_dx(M, N, K)) {
    FewArgs a = few_args(W, dY, *plan, G, set->A, set->stride_a, set->scale, dX, ws, L);
    a.mask = mask;
    a.out_f32 = dX_dtype == WS_DTYPE_F32 ? 1 : 0;
    a.accumulate = (accumulate & WS_ACC_DX) ? 1 : 0;
    WS_RUN(run_few_bwd(a, st));
    return WS_OK;
  }
  const MultiLora ml = multi_of(*plan, ws, L, G, set->A, false, set->stride_a, set->scale);
  WS_RUN(run_nf4_gemm_multi(plan_gemm(true, M, K, N), view(W), dY, M, ml, mask, dX, dX_dtype == WS_DTYPE_F32 ? 1 : 0,
                            (accumulate & WS_ACC_DX) ? 1 : 0, reinterpret_cast<float*>(ws + L.partial), st));
  if (set->n_adapters > kMultiSlots)
    WS_RUN(run_expand(dX_dtype == WS_DTYPE_F32 ? k_multi_expand<false, false, false> : k_multi_expand<false, false, true>,
                      ml, mask, *plan, K, (accumulate & WS_ACC_DX) ? 1 : 0, dX, st));
  return WS_OK;
}

}  // extern "C"
