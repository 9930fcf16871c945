// kv_cache.cu -- the paged cache of keys and values in 8 bits: the plan of a
// step (which rows go where, and how attention's work is shared out), and the
// kernel that appends rows.
//
// A page holds 64 tokens of every kv head.  Its keys [64, D] and its values
// [D, 64] (a token a column: both products of the attention then contract over
// contiguous bytes) are e4m3 codes with one scale each, the smallest power of
// two 2^e with max|x| <= 448 2^e.  Codes are floating-point numbers, so a tight
// scale gains nothing over a power of two, and with powers of two the codes of
// a page whose scale grows keep their values exactly but for those that become
// subnormal: appending token by token is as good as all at once.
#define WS_KV_TU 1
#include <math.h>

#include "kv_plan.cuh"

namespace ws {

cudaError_t kv_cache_read_and_clear_dev_error(uint32_t* flags) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_dev_error, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_dev_error, &zero, sizeof(uint32_t));
}

namespace {

constexpr int kPlanThreads = 1024;

struct KvPlanArgs {
  KvShape s;
  KvLayout L;
  uint8_t* data;
  const int32_t *table, *past, *start;
};

// Exclusive prefix sum of x over the CTA's threads; total to every thread.
WS_DEVINL int block_scan(int x, int* total) {
  __shared__ int part[kPlanThreads / 32 + 1];
  const int lane = (int)lane_id(), w = (int)warp_id();
  int v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();  // part's last readers are through
  if (lane == 31) part[w] = v;
  __syncthreads();
  if (w == 0) {
    int p = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, p, o);
      if (lane >= o) p += y;
    }
    part[lane] = p;
  }
  __syncthreads();
  *total = part[kPlanThreads / 32 - 1];
  return (w ? part[w - 1] : 0) + v - x;
}

// The largest i in [0, n) with at(i) <= x (at(0) <= x; at does not fall).
template <typename F>
WS_DEVINL int last_at_most(int n, int x, F at) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at(mid) <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// One CTA.  Everything read from the caller's arrays is brought into range
// here, and the other kernels go by the plan alone: tokens beyond the table or
// beyond max_new, rows beyond T and pages that are none cannot be reached.
// Bound by latency (prefix sums and searches, one after another): 8 to 11 us for 1
// to 48 sequences, 11 to 12 for 33 with chunks among them, once a step for all layers.
__global__ void __launch_bounds__(kPlanThreads) k_kv_plan(const KvPlanArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int tid = (int)threadIdx.x, n = a.s.n_seq, G = a.s.nh / a.s.nkv;
  KvHeader* hdr = reinterpret_cast<KvHeader*>(a.data);
  int4* seq = reinterpret_cast<int4*>(a.data + a.L.seq);
  int4* pre = reinterpret_cast<int4*>(a.data + a.L.pre);
  int4* append = reinterpret_cast<int4*>(a.data + a.L.append);
  int4* tile = reinterpret_cast<int4*>(a.data + a.L.tile);
  int4* split = reinterpret_cast<int4*>(a.data + a.L.split);
  int* unit = reinterpret_cast<int*>(a.data + a.L.unit);
  int4* c_tile = reinterpret_cast<int4*>(a.data + a.L.c_tile);
  int4* c_split = reinterpret_cast<int4*>(a.data + a.L.c_split);
  int4* c_unit = reinterpret_cast<int4*>(a.data + a.L.c_unit);
  const int room = a.s.max_pages * kPage;

  int n_append = 0, n_tiles = 0, c_tiles = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int s = base + tid;
    int pages = 0, tiles = 0, chunks = 0;
    if (s < n) {
      const int past = min(max(a.past[s], 0), room);
      const int row = min(max(a.start[s], 0), (int)a.s.T);
      const int end = min(max(a.start[s + 1], row), (int)a.s.T);
      const int c = min(min(end - row, a.s.max_new), room - past);
      seq[s] = make_int4(past, row, c, 0);
      if (c > 0) {
        pages = (past + c + kPage - 1) / kPage - past / kPage;
        if (c * G <= kTileRows)
          tiles = 1;
        else
          chunks = (c * G + kChunkRows - 1) / kChunkRows;
      }
    }
    int tp, tt, tc;
    const int p0 = block_scan(pages, &tp), t0 = block_scan(tiles, &tt), c0 = block_scan(chunks, &tc);
    if (s < n) pre[s] = make_int4(n_append + p0, n_tiles + t0, c_tiles + c0, 0);
    n_append += tp;
    n_tiles += tt;
    c_tiles += tc;
  }
  // row ranges that overlap could name more than there is room for
  n_append = min(n_append, (int)a.L.max_append);
  n_tiles = min(n_tiles, (int)a.L.max_tiles);
  c_tiles = min(c_tiles, (int)a.L.c_max_tiles);
  __syncthreads();

  for (int i = tid; i < n_append; i += kPlanThreads) {
    const int s = last_at_most(n, i, [&](int j) { return pre[j].x; });
    const int4 q = seq[s];
    const int p = q.x / kPage + i - pre[s].x;
    const int lo = max(q.x, p * kPage), hi = min(q.x + q.z, (p + 1) * kPage);
    const int page = a.table[(int64_t)s * a.s.max_pages + p];
    append[i] = make_int4(q.y + lo - q.x, page >= 0 ? page : -1, lo - p * kPage, hi - lo);
  }

  // ---- decode: one tile a sequence
  int W = 0;
  for (int base = 0; base < n_tiles; base += kPlanThreads) {
    const int i = base + tid;
    int pages = 0, s = 0;
    if (i < n_tiles) {
      s = last_at_most(n, i, [&](int j) { return pre[j].y; });
      pages = (seq[s].x + seq[s].z - 1) / kPage + 1;
    }
    int total;
    const int at = block_scan(pages, &total);
    if (i < n_tiles) tile[i] = make_int4(s, 0, W + at, -1);
    W += total;
  }
  if (tid == 0) tile[n_tiles] = make_int4(0, 0, W, -1);
  __syncthreads();

  const int U = max(1, min((int)a.L.max_units, W));
  int n_split = 0;
  for (int base = 0; base < n_tiles; base += kPlanThreads) {
    const int i = base + tid;
    int u0 = 0, u1 = 0;
    if (i < n_tiles) {
      u0 = unit_of(tile[i].z, W, U);
      u1 = unit_of(tile[i + 1].z - 1, W, U);
    }
    int total;
    const int j = n_split + block_scan(u1 > u0, &total);
    if (u1 > u0) {
      tile[i].w = j;
      // slot = unit + index among the cut tiles: no two pieces share one
      split[2 * j] = make_int4(u0 + j, u1 - u0 + 1, 0, 0);
      split[2 * j + 1] = seq[tile[i].x];
    }
    n_split += total;
  }
  if (n_tiles > 0)
    for (int u = tid; u < U; u += kPlanThreads)
      unit[u] = last_at_most(n_tiles, (int)unit_start(u, W, U), [&](int j) { return tile[j].z; });

  // ---- chunk: 256-row tiles, shares of all heads' steps
  // A tile's cost is kChunkTileCost and its steps, or half of those where both slots share them (tiles of up to
  // half the rows).  A share that would begin in the first part begins with the tile.
  auto halved = [](int rows) { return rows <= kChunkRows / 2; };
  auto opening = [](bool half) { return half ? kChunkHalfTileCost : kChunkTileCost; };
  int Wc = 0, cost = 0;
  for (int base = 0; base < c_tiles; base += kPlanThreads) {
    const int i = base + tid;
    int steps = 0, s = 0, r0 = 0, mine = 0;
    if (i < c_tiles) {
      s = last_at_most(n, i, [&](int j) { return pre[j].z; });
      r0 = (i - pre[s].z) * kChunkRows;
      const int rows = min(seq[s].z * G - r0, kChunkRows);
      steps = (seq[s].x + (r0 + rows - 1) / G) / (2 * kPage) + 1;
      mine = opening(halved(rows)) + (halved(rows) ? (steps + 1) / 2 : steps);
    }
    int total, all;
    const int at = block_scan(steps, &total), before = block_scan(mine, &all);
    if (i < c_tiles) c_tile[i] = make_int4(s, r0, Wc + at, cost + before);
    Wc += total;
    cost += all;
  }
  if (tid == 0) c_tile[c_tiles] = make_int4(0, 0, Wc, cost);
  __syncthreads();
  int Uc = 0, n_cut = 0;
  if (c_tiles > 0) {
    const int64_t all = (int64_t)cost * a.s.nkv;
    Uc = (int)max((int64_t)1, min(a.L.c_max_units, all / kChunkMinSteps));
    // a unit's start cuts a (head, tile) pair, or lies between two; units that start in one pair come together
    for (int base = 0; base <= Uc; base += kPlanThreads) {
      const int u = base + tid;
      int t = 0, h = a.s.nkv, step = 0;
      bool first = false;
      if (u < Uc) {
        const int64_t x = unit_start(u, all, Uc);
        h = (int)(x / cost);
        const int y = (int)(x % cost);
        t = last_at_most(c_tiles, y, [&](int j) { return c_tile[j].w; });
        const bool half = halved(seq[c_tile[t].x].z * G - c_tile[t].y);
        const int open = c_tile[t].w + opening(half);
        step = max(y - open, 0) << half;
        first = step > 0 && unit_start(u - 1, all, Uc) <= (int64_t)h * cost + open;
      }
      int total;
      const int j = n_cut + block_scan(first, &total);
      if (u <= Uc) c_unit[u] = make_int4(t, h, step > 0 ? (first ? j : j - 1) : -1, step);
      if (first) {
        const int64_t end = (int64_t)h * cost + c_tile[t + 1].w;
        c_split[2 * j] = make_int4(u - 1 + j, unit_of(end - 1, all, Uc) - (u - 1) + 1, c_tile[t].y, h);
        c_split[2 * j + 1] = seq[c_tile[t].x];
      }
      n_cut += total;
    }
  }
  if (tid == 0) {
    hdr->n_append = n_append;
    hdr->n_tiles = n_tiles;
    hdr->pages = W;
    hdr->units = n_tiles > 0 ? U : 0;
    hdr->n_split = n_split;
    hdr->c_tiles = c_tiles;
    hdr->c_steps = Wc;
    hdr->c_units = Uc;
    hdr->c_split = n_cut;
    hdr->sig[0] = a.L.sig[0];
    hdr->sig[1] = a.L.sig[1];
  }
}

// ---- append ------------------------------------------------------------------------
struct AppendArgs {
  uint8_t *k, *v;
  float* scale;
  const uint8_t* plan;
  size_t off_append;
  uint32_t sig[2];
  const uint16_t *xk, *xv;
  int64_t sk, sv, n_pages;
  int nkv;
};

// The codes of a word again, for a scale 1/ratio times theirs.
WS_DEVINL uint32_t rescale4(uint32_t w, float ratio) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float lo, hi;
    e4m3x2_values((w >> (16 * i)) & 0xffffu, lo, hi);
    out |= e4m3x2(lo * ratio, hi * ratio) << (16 * i);
  }
  return out;
}
// The scale for values up to `top` (bf16 bits without the sign): 2^e with the
// smallest e >= -126 such that top <= 448 2^e; NaN where top is not finite.
WS_DEVINL float scale_for(uint32_t top) {
  if (top >= 0x7f80u) return __uint_as_float(0x7fc00000u);
  // 448 = 1.75 2^8: one exponent more where the mantissa is above 1.75
  const int e = (int)(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u);
  return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}
// A page that goes on from place `lo` and turns NaN keeps in the NaN what it was: the exponent of its scale, and lo, from
// which on its codes are zero.  Going on from there or before, those that were not finite having been taken back, gives
// the scale again.  Bits 14 to 21 tell such a NaN from others.
constexpr uint32_t kNan = 0x7fc00000u, kNanMark = kNan | 0xa5u << 14;
WS_DEVINL float nan_of(float scale, int lo) {
  const uint32_t b = __float_as_uint(scale);
  if (isnan(scale)) return scale;
  return __uint_as_float(lo > 0 && (b & 0x807fffffu) == 0u ? kNanMark | (b >> 23) << 6 | (uint32_t)lo : kNan);
}
// The scale of a page that goes on from place lo.
WS_DEVINL float scale_at(float scale, int lo) {
  const uint32_t b = __float_as_uint(scale);
  return (b & ~0x3fffu) == kNanMark && lo <= (int)(b & 63u) ? __uint_as_float((b >> 6 & 0xffu) << 23) : scale;
}
WS_DEVINL uint32_t max_abs(const uint4& w, uint32_t m) {
  m = __vmaxu2(m, w.x & 0x7fff7fffu);
  m = __vmaxu2(m, w.y & 0x7fff7fffu);
  m = __vmaxu2(m, w.z & 0x7fff7fffu);
  return __vmaxu2(m, w.w & 0x7fff7fffu);
}
WS_DEVINL float elem(const uint4& w, int i) {  // element i of eight
  const uint32_t x = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
  return (i & 1) ? bf16_hi(x) : bf16_lo(x);
}

// One CTA per (touched page, kv head).  Thread (c, t) has elements 8c .. 8c + 7
// of the page's tokens 8t .. 8t + 7: rows come in 16-byte pieces, key codes
// leave in 8-byte pieces of whole rows, value codes are turned round through
// shared memory.  Bound by memory for prompts (3 bytes an element: eight prompts,
// 22600 rows of 8 heads of 128, in 27 us, 5.2 TB/s), by the latency of three
// dependent loads and the launch for single tokens (48 rows: 6 us in a stream).
template <int D>
__global__ void __launch_bounds__(D) k_kv_append(const AppendArgs a) {
  constexpr int C = D / 8;  // pieces of a row; D = C * 8 threads
  __shared__ __align__(16) uint8_t vt[D * kPage];
  __shared__ uint32_t top[2][D / 32];
  pdl_wait();
  pdl_launch_dependents();
  if (!plan_filled_or_say(a.plan, a.sig)) return;
  const int item = (int)blockIdx.x / a.nkv, head = (int)blockIdx.x % a.nkv;
  if (item >= reinterpret_cast<const KvHeader*>(a.plan)->n_append) return;
  const int4 it = reinterpret_cast<const int4*>(a.plan + a.off_append)[item];
  if (it.y < 0 || it.y >= a.n_pages) return;
  const int tid = (int)threadIdx.x, c = tid % C, t = tid / C;
  const int lo = it.z, hi = it.z + it.w;  // the new tokens' places
  const int64_t at = (int64_t)it.y * a.nkv + head;
  uint8_t* pk = a.k + at * (kPage * D);
  uint8_t* pv = a.v + at * (kPage * D);
  float2* ps = reinterpret_cast<float2*>(a.scale) + at;
  float2 old = lo > 0 ? *ps : make_float2(0.0f, 0.0f);
  old = make_float2(scale_at(old.x, lo), scale_at(old.y, lo));

  uint4 xk[8], xv[8];
  uint32_t mk = 0, mv = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int p = 8 * t + i;
    xk[i] = xv[i] = make_uint4(0, 0, 0, 0);
    if (p >= lo && p < hi) {
      const int64_t row = it.x + p - lo;
      xk[i] = *reinterpret_cast<const uint4*>(a.xk + row * a.sk + head * D + c * 8);
      xv[i] = *reinterpret_cast<const uint4*>(a.xv + row * a.sv + head * D + c * 8);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    mk = max_abs(xk[i], mk);
    mv = max_abs(xv[i], mv);
  }
  mk = __reduce_max_sync(0xffffffffu, max(mk & 0xffffu, mk >> 16));
  mv = __reduce_max_sync(0xffffffffu, max(mv & 0xffffu, mv >> 16));
  if (lane_id() == 0) {
    top[0][warp_id()] = mk;
    top[1][warp_id()] = mv;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    mk = max(mk, top[0][w]);
    mv = max(mv, top[1][w]);
  }
  // a page that goes on keeps a scale no smaller than it had, NaN included
  float ks = scale_for(mk), vs = scale_for(mv);
  if (isnan(ks))
    ks = nan_of(old.x, lo);
  else if (lo > 0 && !(old.x <= ks))
    ks = old.x;
  if (isnan(vs))
    vs = nan_of(old.y, lo);
  else if (lo > 0 && !(old.y <= vs))
    vs = old.y;
  const bool grow_k = lo > 0 && ks > old.x, grow_v = lo > 0 && vs > old.y;
  // codes under a NaN scale are zero: a code that is NaN would reach rows that do not see it, as 0 * NaN
  const bool bad_k = isnan(ks), bad_v = isnan(vs);
  const float ik = 1.0f / ks, iv = 1.0f / vs;

#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int p = 8 * t + i;
    uint2* dst = reinterpret_cast<uint2*>(pk + p * D + c * 8);
    if (p >= lo && p < hi) {
      uint32_t w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w[j] = e4m3x2(elem(xk[i], 4 * j) * ik, elem(xk[i], 4 * j + 1) * ik) |
               e4m3x2(elem(xk[i], 4 * j + 2) * ik, elem(xk[i], 4 * j + 3) * ik) << 16;
      *dst = bad_k ? make_uint2(0, 0) : make_uint2(w[0], w[1]);
    } else if (grow_k && p < lo) {
      const uint2 o = *dst;
      *dst = make_uint2(rescale4(o.x, old.x * ik), rescale4(o.y, old.x * ik));
    }
  }
  // Values: row d of [D][64] in shared memory, its 8-byte units at unit ^ (d / 8)
  // % 8, so that a half warp's 16 rows meet in pairs only.
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[h] = e4m3x2(elem(xv[4 * h], j) * iv, elem(xv[4 * h + 1], j) * iv) |
             e4m3x2(elem(xv[4 * h + 2], j) * iv, elem(xv[4 * h + 3], j) * iv) << 16;
    *reinterpret_cast<uint2*>(vt + (8 * c + j) * kPage + ((t ^ (c & 7)) << 3)) =
        bad_v ? make_uint2(0, 0) : make_uint2(w[0], w[1]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // D * 4 pieces of 16 tokens
    const int d = (tid + i * D) / 4, u = (tid + i * D) % 4, f = 16 * u, x = (d / 8) & 7;
    if (!(f < hi && f + 16 > lo) && !(grow_v && f < lo)) continue;
    const uint2 n0 = *reinterpret_cast<const uint2*>(vt + d * kPage + (((2 * u) ^ x) << 3));
    const uint2 n1 = *reinterpret_cast<const uint2*>(vt + d * kPage + (((2 * u + 1) ^ x) << 3));
    uint32_t w[4] = {n0.x, n0.y, n1.x, n1.y};
    uint4* dst = reinterpret_cast<uint4*>(pv + d * kPage + f);
    if (lo > f || hi < f + 16) {  // others' places in it
      const uint4 o4 = *dst;
      const uint32_t o[4] = {o4.x, o4.y, o4.z, o4.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int b = f + 4 * j;  // first token of the word
        const uint32_t older = grow_v && b < lo ? rescale4(o[j], old.y * iv) : o[j];
        uint32_t keep = 0, mine = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (b + e < lo) keep |= 0xffu << (8 * e);
          if (b + e >= lo && b + e < hi) mine |= 0xffu << (8 * e);
        }
        w[j] = (older & keep) | (w[j] & mine) | (o[j] & ~(keep | mine));
      }
    }
    *dst = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (tid == 0) *ps = make_float2(ks, vs);
}

bool al16k(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al4k(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

ws_status kv_shape(const ws_kv_plan* p, KvShape* s) {
  if (!p) return WS_ERR_INVALID;
  if (p->n_seq < 1 || p->n_seq > WS_KV_MAX_SEQS || p->max_pages < 1 || p->max_pages > 1 << 20 ||
      (int64_t)p->n_seq * p->max_pages > (int64_t)1 << 28)
    return WS_ERR_SHAPE;
  if (p->T < 1 || p->T > (int64_t)1 << 20 || p->max_new < 1 || p->max_new > p->T) return WS_ERR_SHAPE;
  if (p->n_kv_heads < 1 || p->n_kv_heads > 256 || p->n_heads < 1 || p->n_heads > 1024 ||
      p->n_heads % p->n_kv_heads)
    return WS_ERR_SHAPE;
  if (p->head_dim != 64 && p->head_dim != 128) return WS_ERR_SHAPE;
  *s = KvShape{p->T, p->n_seq, p->max_pages, p->max_new, p->n_heads, p->n_kv_heads, p->head_dim};
  // the chunk kernel's shares count one head's cost in 32 bits, all heads' in 64
  const int64_t cost = kv_chunk_tiles(*s) * (s->max_pages / 2 + 1 + kChunkTileCost);
  if (cost > 0x7fffffff || cost * s->nkv > (int64_t)1 << 36) return WS_ERR_SHAPE;
  return WS_OK;
}
ws_status kv_check(const ws_kv_cache* c, const ws_kv_plan* p, KvShape* s) {
  const ws_status st = kv_shape(p, s);
  if (st != WS_OK) return st;
  if (!c || !c->k || !c->v || !c->scale || !p->data || !p->page_table) return WS_ERR_INVALID;
  if (c->n_pages < 1 || c->n_pages > 0x7fffffff / s->nkv || c->n_kv_heads != s->nkv || c->head_dim != s->hd)
    return WS_ERR_SHAPE;
  if (!al16k(c->k) || !al16k(c->v) || !al16k(c->scale) || !al16k(p->data) || !al4k(p->page_table))
    return WS_ERR_ALIGN;
  return WS_OK;
}

}  // namespace ws

using namespace ws;

extern "C" {

ws_status ws_kv_plan_size(const ws_kv_plan* plan, size_t* bytes) {
  KvShape s;
  const ws_status st = kv_shape(plan, &s);
  if (st != WS_OK) return st;
  if (!bytes) return WS_ERR_INVALID;
  *bytes = kv_layout(s).bytes;
  return WS_OK;
}

ws_status ws_kv_plan_init(const ws_kv_plan* plan, const int32_t* past, const int32_t* row_start,
                          ws_stream_t stream) {
  KvPlanArgs a;
  const ws_status st = kv_shape(plan, &a.s);
  if (st != WS_OK) return st;
  if (!plan->data || !plan->page_table || !past || !row_start) return WS_ERR_INVALID;
  if (!al16k(plan->data) || !al4k(plan->page_table) || !al4k(past) || !al4k(row_start)) return WS_ERR_ALIGN;
  a.L = kv_layout(a.s);
  a.data = static_cast<uint8_t*>(plan->data);
  a.table = plan->page_table;
  a.past = past;
  a.start = row_start;
  note_launch();
  const cudaError_t e = launch_pdl(k_kv_plan, dim3(1), dim3(kPlanThreads), 0, (cudaStream_t)stream, a);
  return e == cudaSuccess ? WS_OK : WS_ERR_CUDA;
}

ws_status ws_kv_append(const ws_kv_cache* cache, const ws_kv_plan* plan, const uint16_t* k,
                       int64_t k_stride, const uint16_t* v, int64_t v_stride, ws_stream_t stream) {
  KvShape s;
  const ws_status st = kv_check(cache, plan, &s);
  if (st != WS_OK) return st;
  if (!k || !v) return WS_ERR_INVALID;
  for (int64_t d : {k_stride, v_stride})
    if (d < (int64_t)s.nkv * s.hd || d % 8 || d > (int64_t)1 << 31) return WS_ERR_SHAPE;
  if (!al16k(k) || !al16k(v)) return WS_ERR_ALIGN;
  const KvLayout L = kv_layout(s);
  AppendArgs a;
  a.k = cache->k;
  a.v = cache->v;
  a.scale = cache->scale;
  a.plan = static_cast<const uint8_t*>(plan->data);
  a.off_append = L.append;
  a.sig[0] = L.sig[0];
  a.sig[1] = L.sig[1];
  a.xk = k;
  a.xv = v;
  a.sk = k_stride;
  a.sv = v_stride;
  a.n_pages = cache->n_pages;
  a.nkv = s.nkv;
  note_launch();
  const cudaError_t e = launch_pdl(s.hd == 64 ? k_kv_append<64> : k_kv_append<128>,
                                   dim3((unsigned)(L.max_append * s.nkv)), dim3((unsigned)s.hd), 0,
                                   (cudaStream_t)stream, a);
  return e == cudaSuccess ? WS_OK : WS_ERR_CUDA;
}

}  // extern "C"
