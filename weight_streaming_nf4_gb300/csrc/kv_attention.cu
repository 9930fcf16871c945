// kv_attention.cu -- attention over the paged 8-bit cache.
//
// New row i of a sequence with `past` tokens in the cache before the call sees
// tokens 0 .. past + i.  Query head h reads kv head h / G, G = n_heads /
// n_kv_heads; a sequence's rows for one kv head are its (new token, head of the
// group) pairs, R = i G + h % G, so a group's heads share what is read.
//
// Decoding rows (k_kv_decode; sequences of more than kTileRows rows go to
// kv_chunk.cu: a second tile of 16 would read the codes again.  24 sequences of
// 2400 to 16000 tokens, 240k in all, 40 + 8 heads: 123 us with 15 rows each here,
// 157 with 20 there).  Bound by memory: each code is read once.  One
// warp has a contiguous share of the pages of all 16-row tiles (equal shares,
// so ragged batches fill the device), copies a page's keys and values (8 KB
// each at D = 128) into shared memory while the ones before are used, and joins
// its pages with a running maximum and sum (Milakov and Gimelshein, 2018).  Both products are the small-tile
// tensor operation m16n8k16 in fp16, which holds e4m3 codes exactly:
//   S^T = K Q^T  (16 tokens x 8 rows),   O^T += V^T P^T  (16 elements x 8 rows).
// The contraction may run in any order, so a thread takes 32 (D = 64: 16)
// neighbouring bytes of a key row, and 16 neighbouring tokens of a value row,
// as its share of the operand: wide loads, one conversion a pair of codes, no
// exchange but a transposition of P in registers (movmatrix).  Which token is
// which row of S^T is chosen so that P arrives where V^T wants it.
// Queries enter as fp16 times a power of two of their row, values' scales go
// into P (page_ref in kv_plan.cuh), keys' scales into the exponent.
// P enters as two fp16 numbers, what one leaves being the other: 2^-22 of itself
// for the 2^-11 of one, which is what results of terms that cancel are off by.
// The second product's operations double; the pages' way stays what bounds it.
// A page's products are summed by themselves and then added to O: the tensor
// cores' additions cut off instead of rounding, up to 2^-23 of the sum each time,
// and over a share of 128 pages would lose 2^-16 of its sizes, always the same way.
// (Free for up to eight rows; for sixteen, whose registers are all in use, 4 us of
// the 64 below.)
// Tiles cut by a share's end are joined by k_kv_join, in a fixed order.
// Where no tile of the plan can have more than eight rows, NQ = 1 leaves the
// second half of the operands out (188 registers for 255).
// 48 sequences of 2400 to 16000 tokens, 479k in all, 40 + 8 heads of 128: 158 us
// with the join, 6.2 TB/s (0.92 of the copy rate).  Two of 130000 and 85000, 28 + 4
// heads, two new tokens each: 64 us, 3.4 TB/s: a share is 11 pages, so start, ramp
// and partial results are a quarter, and 14 rows of P in two parts take four tensor
// operations where up to eight rows in one part take one (53 us with one part, summed
// in the tensor cores).
#define WS_KV_TU 1
#include <math.h>

#include "kv_plan.cuh"

namespace ws {

cudaError_t kv_read_and_clear_dev_error(uint32_t* flags) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_dev_error, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_dev_error, &zero, sizeof(uint32_t));
}

namespace {

constexpr int kDecodeWarps = 4;
constexpr int kPMargin = 14;  // P in [0, 1] times 2^14, so that small ones keep bits in fp16

WS_DEVINL void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
WS_DEVINL uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// 2^e for the fp32 bits' exponent of a finite x > 0 brought to e <= 126.
WS_DEVINL float q_scale(float top) {
  // top 2^k in [2^14, 2^15): fp16 keeps bf16's bits down to 2^-28 of the row's largest
  const int e = (int)(__float_as_uint(top) >> 23) - 127;
  return __uint_as_float((uint32_t)(min(kPMargin - e, 126) + 127) << 23);
}

template <int D>
struct DecodeSmem {
  static constexpr uint32_t PAGE = kPage * D;      // bytes of a page's keys, or values
  static constexpr int RING = 3;                   // a warp's copies: keys, values, keys, ... in turn
  static constexpr uint32_t OFF_BAR = kDecodeWarps * RING * PAGE;
  static constexpr uint32_t BYTES = OFF_BAR + kDecodeWarps * RING * 8 + 128;
  static constexpr int CTAS = decode_warps(D) / kDecodeWarps;  // an SM
};

// A page of a tile on a warp's way: what it takes to load and to use it.
struct Step {
  int tile, p, pend;  // page p of the tile; the warp's share of the tile ends at pend
  int page;           // its place in the cache, -1: none
  float ks, vs;
  int seq;
};

template <int D, int NQ>
__global__ void __launch_bounds__(kDecodeWarps * 32, DecodeSmem<D>::CTAS) k_kv_decode(const __grid_constant__ KvAttnArgs a) {
  using L = DecodeSmem<D>;
  constexpr int KS = D / 16;   // contraction steps of S
  constexpr int HT = D / 16;   // 16-element tiles of O
  constexpr int KW = D / 64;   // 16-byte pieces a thread has of a key row
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const int warp = (int)warp_id(), lane = (int)lane_id(), g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * (L::RING * L::PAGE);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR) + L::RING * warp;
  if (lane == 0) {
    for (int i = 0; i < L::RING; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
  }
  __syncwarp();
  pdl_wait();
  pdl_launch_dependents();
  if (*(volatile uint32_t*)&g_dev_error != 0u || !plan_filled_or_say(a.plan, a.L.sig)) return;

  const KvHeader* hdr = reinterpret_cast<const KvHeader*>(a.plan);
  const int4* tiles = reinterpret_cast<const int4*>(a.plan + a.L.tile);
  const int4* seqs = reinterpret_cast<const int4*>(a.plan + a.L.seq);
  const int W = hdr->pages, U = hdr->units;
  const int w = (int)blockIdx.x * kDecodeWarps + warp;
  const int head = w % a.nkv, u = w / a.nkv;
  if (u >= U) return;
  const int begin = (int)unit_start(u, W, U), end = (int)unit_start(u + 1, W, U);

  // The steps: pages begin .. end - 1 of the tiles' pages behind one another.
  auto fill = [&](Step& s) {
    s.ks = s.vs = 0.0f;
    s.page = a.table[(int64_t)s.seq * a.max_pages + s.p];
    if (s.page < 0 || s.page >= a.n_pages) {
      s.page = -1;
      return;
    }
    const float2 sc = *(reinterpret_cast<const float2*>(a.scale) + (int64_t)s.page * a.nkv + head);
    s.ks = sc.x;
    s.vs = sc.y;
  };
  auto enter = [&](Step& s, int tile) {  // a tile's first page in this share
    const int4 tl = tiles[tile];
    s.tile = tile;
    s.seq = tl.x;
    s.p = max(begin, tl.z) - tl.z;
    s.pend = min(end, tiles[tile + 1].z) - tl.z;
  };
  auto follow = [&](Step& s) {  // the step behind s, none: pend 0
    if (s.p + 1 < s.pend) {
      ++s.p;
    } else if (tiles[s.tile + 1].z < end) {
      enter(s, s.tile + 1);
    } else {
      s.pend = 0;
      s.page = -1;
      return;
    }
    fill(s);
  };
  // Copies go round the ring; a page that is none completes its turn at once.
  int in = 0, out = 0;            // ring places of the next copy, and of the next to be used
  uint32_t out_ph = 0;
  auto load = [&](const Step& s, bool values) {
    if (s.pend == 0) return;
    if (lane == 0) {
      if (s.page < 0) {
        mbar_arrive(&bars[in]);
      } else {
        const int64_t at = ((int64_t)s.page * a.nkv + head) * L::PAGE;
        mbar_arrive_expect_tx(&bars[in], L::PAGE);
        bulk_load(ring + in * L::PAGE, (values ? a.v : a.k) + at, L::PAGE, &bars[in]);
      }
    }
    in = in == L::RING - 1 ? 0 : in + 1;
  };
  // The next copy has come.  Where it does not, the others in flight are waited for.
  auto take = [&]() {
    if (__all_sync(0xffffffffu, mbar_wait(&bars[out], out_ph, DERR_TIMEOUT_FULL))) return true;
    for (int i = 1; i < L::RING; ++i) {
      const int b = (out + i) % L::RING;
      mbar_wait(&bars[b], out + i >= L::RING ? out_ph ^ 1u : out_ph, DERR_TIMEOUT_DRAIN);
    }
    return false;
  };
  auto next_place = [&]() {
    out = out == L::RING - 1 ? 0 : out + 1;
    out_ph ^= out == 0;
  };
  Step cur, nxt, nx2;
  enter(cur, reinterpret_cast<const int*>(a.plan + a.L.unit)[u]);
  fill(cur);
  nxt = cur;
  follow(nxt);
  load(cur, false);
  load(cur, true);
  load(nxt, false);
  bool fresh = true;

  uint32_t bq[NQ][KS][2];          // Q^T operands
  float o[NQ][HT][4];              // O^T, sums over the pages so far: elements 16 ht + g (+ 8), rows 8 nq + 2t (+ 1)
  float m[NQ][2], l[NQ][2], ref[NQ][2], qs[NQ][2];
  int lim[NQ][2];                  // tokens each row sees
  int rows = 0, kv_end = 0, first_lim = 0;
  bool wide = false;               // more than eight rows: the second half of the operands is in use
  int4 tl = make_int4(0, 0, 0, 0), sq = tl;

  for (; cur.pend != 0; cur = nxt, nxt = nx2) {
    const bool last = cur.p + 1 == cur.pend;
    nx2 = nxt;
    if (nxt.pend != 0) follow(nx2);
    if (fresh) {
      tl = tiles[cur.tile];
      sq = seqs[cur.seq];
      rows = sq.z * a.G;
      wide = rows > 8;
      kv_end = sq.x + sq.z;
      first_lim = sq.x + 1;
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) {
        // row 8 nq + g: elements D/4 t .. of it
        const int r = 8 * nq + g;
        uint4 x[2 * KW];
#pragma unroll
        for (int i = 0; i < 2 * KW; ++i) x[i] = make_uint4(0, 0, 0, 0);
        if (r < rows) {
          const int i = r / a.G;
          const uint16_t* src = a.q + (int64_t)(sq.y + i) * a.sq + (head * a.G + r - i * a.G) * D + t * (D / 4);
#pragma unroll
          for (int j = 0; j < 2 * KW; ++j) x[j] = *reinterpret_cast<const uint4*>(src + 8 * j);
        }
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 2 * KW; ++j) {
          top = __vmaxu2(top, __vmaxu2(x[j].x & 0x7fff7fffu, x[j].y & 0x7fff7fffu));
          top = __vmaxu2(top, __vmaxu2(x[j].z & 0x7fff7fffu, x[j].w & 0x7fff7fffu));
        }
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float qk = q_scale(__uint_as_float(top << 16));
#pragma unroll
        for (int j = 0; j < 2 * KW; ++j) {
          const uint32_t e[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            bq[nq][2 * j + (i >> 1)][i & 1] = pack_f16x2(bf16_lo(e[i]) * qk, bf16_hi(e[i]) * qk);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = 2 * t + e;  // the row of this thread's columns of S^T
          qs[nq][e] = a.sl2 / __shfl_sync(0xffffffffu, qk, 4 * c);
          lim[nq][e] = 8 * nq + c < rows ? sq.x + (8 * nq + c) / a.G + 1 : 0;
          m[nq][e] = ref[nq][e] = -INFINITY;
          l[nq][e] = 0.0f;
        }
#pragma unroll
        for (int ht = 0; ht < HT; ++ht)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nq][ht][e] = 0.0f;
      }
    }

    if (!take()) return;
    if (cur.page >= 0) {
      const uint8_t* sk = ring + out * L::PAGE;
      // S^T.  Row r of block b (8 rows) is token 16 (r / 2) + 2 b + r % 2.
      float s[NQ][4][4];
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        uint4 k0[KW], k1[KW];
        const uint8_t* row = sk + (16 * (g >> 1) + 4 * mt + (g & 1)) * D + t * (D / 4);
#pragma unroll
        for (int j = 0; j < KW; ++j) {
          k0[j] = *reinterpret_cast<const uint4*>(row + 16 * j);
          k1[j] = *reinterpret_cast<const uint4*>(row + 2 * D + 16 * j);
        }
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nq][mt][e] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint4 &w0 = k0[ks >> 2], &w1 = k1[ks >> 2];
          const int i = ks & 3;
          uint32_t a0, a1, a2, a3;
          decode4(i == 0 ? w0.x : i == 1 ? w0.y : i == 2 ? w0.z : w0.w, a0, a2);
          decode4(i == 0 ? w1.x : i == 1 ? w1.y : i == 2 ? w1.z : w1.w, a1, a3);
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq)
            if (nq == 0 || wide) mma_f16(s[nq][mt], a0, a1, a2, a3, bq[nq][ks][0], bq[nq][ks][1]);
        }
      }
      __syncwarp();
      next_place();
      load(nxt, true);

      // softmax: columns (rows of q) 2t, 2t + 1; tokens 16 (g / 2) + 4 mt + g % 2 (+ 2)
      const int tok0 = cur.p * kPage + 16 * (g >> 1) + (g & 1);
      const bool tail = (cur.p + 1) * kPage > first_lim;
      float vf;  // NaN for a page that holds one
      const float ve = scale_parts(cur.vs, vf);
      uint32_t bp[NQ][4][2], br[NQ][4][2];  // P as fp16 and the rest
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) {
        if (nq > 0 && !wide) break;
        float nm[2], nr[2], cf[2], vr[2];
        if (tail) {
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (tok0 + 4 * mt + 2 * (i >> 1) >= lim[nq][i & 1]) s[nq][mt][i] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float c = qs[nq][e] * cur.ks;
          cf[e] = c < 1e-37f ? 1e-37f : c;  // not below fp32's range: -inf * 0 is NaN
          float top = -INFINITY;
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) top = fmaxf(top, fmaxf(s[nq][mt][e], s[nq][mt][2 + e]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          top *= cf[e];
          nm[e] = fmaxf(m[nq][e], top);
          // (infinities of one sign give NaN, which the maximum passes over)
          nr[e] = fmaxf(floorf(ref[nq][e] + (m[nq][e] - nm[e])), page_ref(top - nm[e], ve));
          vr[e] = page_factor(ve, nr[e], (float)kPMargin) * vf;
        }
        const bool moved = nm[0] != m[nq][0] || nm[1] != m[nq][1] || nr[0] != ref[nq][0] || nr[1] != ref[nq][1];
        if (__any_sync(0xffffffffu, moved)) {
          float c[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float d = m[nq][e] - nm[e], dr = ref[nq][e] - nr[e];
            l[nq][e] *= nm[e] == -INFINITY ? 1.0f : ex2(d);
            c[e] = nm[e] == -INFINITY ? 1.0f : ex2(d + dr);
            m[nq][e] = nm[e];
            ref[nq][e] = nr[e];
          }
#pragma unroll
          for (int ht = 0; ht < HT; ++ht)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nq][ht][e] *= c[e & 1];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float base = nm[e] == -INFINITY ? 0.0f : nm[e];
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float& x = s[nq][mt][2 * h + e];
              x = ex2(fmaf(x, cf[e], -base));
            }
        }
        if (tail) {  // a row gets none of the scales of a page that it does not see, NaN included
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (tok0 + 4 * mt + 2 * (i >> 1) >= lim[nq][i & 1]) s[nq][mt][i] = 0.0f;
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            l[nq][i & 1] += s[nq][mt][i];
            s[nq][mt][i] *= vr[i & 1];
          }
        if (tail) {
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (tok0 + 4 * mt + 2 * (i >> 1) >= lim[nq][i & 1]) s[nq][mt][i] = 0.0f;
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t hi, rest;
            split_f16x2(s[nq][mt][2 * h], s[nq][mt][2 * h + 1], hi, rest);
            bp[nq][mt][h] = transpose8x8(hi);
            br[nq][mt][h] = transpose8x8(rest);
          }
      }

      if (!take()) return;
      const uint8_t* sv = ring + out * L::PAGE;
      // places behind the last token hold anything: P is zero there, and a code could be NaN
      const int left = kv_end - cur.p * kPage - 16 * t;
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        uint4 v0 = *reinterpret_cast<const uint4*>(sv + (16 * ht + g) * kPage + 16 * t);
        uint4 v1 = *reinterpret_cast<const uint4*>(sv + (16 * ht + g + 8) * kPage + 16 * t);
        uint32_t x0[4] = {v0.x, v0.y, v0.z, v0.w}, x1[4] = {v1.x, v1.y, v1.z, v1.w};
        if (tail) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = left - 4 * i;
            const uint32_t keep = n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
            x0[i] &= keep;
            x1[i] &= keep;
          }
        }
        float add[NQ][4];
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
          for (int e = 0; e < 4; ++e) add[nq][e] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a0, a1, a2, a3;
          decode4(x0[i], a0, a2);
          decode4(x1[i], a1, a3);
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq)
            if (nq == 0 || wide) {
              mma_f16(add[nq], a0, a1, a2, a3, bp[nq][i][0], bp[nq][i][1]);
              mma_f16(add[nq], a0, a1, a2, a3, br[nq][i][0], br[nq][i][1]);
            }
        }
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nq][ht][e] += add[nq][e];
      }
      __syncwarp();
      next_place();
      load(nx2, false);
    } else {
      next_place();
      load(nxt, true);
      if (!take()) return;
      next_place();
      load(nx2, false);
    }

    fresh = last;
    if (!last) continue;
    // the tile's end in this share
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nq][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const bool none = sum == 0.0f;
        const float f = (1.0f / (1 << kPMargin)) / sum, g2 = pow2(ref[nq][e]);
        const float lse2 = none ? -INFINITY : m[nq][e] + log2f(sum);
        const int r = 8 * nq + 2 * t + e;
        if (r >= rows) continue;
        if (tl.w < 0) {
          const int i = r / a.G, h = head * a.G + r - i * a.G;
          uint16_t* dst = a.o + (int64_t)(sq.y + i) * a.so + h * D;
#pragma unroll
          for (int ht = 0; ht < HT; ++ht) {
            dst[16 * ht + g] = f32_to_bf16_bits(none ? 0.0f : o[nq][ht][e] * f * g2);
            dst[16 * ht + g + 8] = f32_to_bf16_bits(none ? 0.0f : o[nq][ht][2 + e] * f * g2);
          }
          if (a.lse && g == 0) a.lse[(int64_t)h * a.T + sq.y + i] = lse2 * kLn2;
        } else {
          const int64_t at = ((int64_t)(u + tl.w) * a.nkv + head) * kTileRows + r;
          float* dst = a.part_o + at * D;
#pragma unroll
          for (int ht = 0; ht < HT; ++ht) {
            dst[16 * ht + g] = none ? 0.0f : o[nq][ht][e] * f * g2;
            dst[16 * ht + g + 8] = none ? 0.0f : o[nq][ht][2 + e] * f * g2;
          }
          if (g == 0) a.part_l[at] = lse2;
        }
      }
  }
}

// Cut tiles: row r's pieces o_i with log2-sums l_i are sum 2^(l_i) o_i / sum 2^(l_i).
// Few pieces (decode batches): a warp a row, all rows in one CTA.  Many (contexts of
// 130000 and 85000 tokens leave 185 and 121 a row): a CTA a row, its warps taking every
// sixteenth piece.  Sums have a fixed order.  Bound by latency: what it takes to
// know where to look is one trip to memory, and CTAs that find nothing there leave
// the sooner the more fit on an SM.  Four pieces in flight a warp and two CTAs an
// SM: the 48 sequences above take 158 us in all, the two 64; eight and one CTA 162
// and 63.
constexpr int kJoinWarps = 16, kJoinFlight = 4, kJoinFew = 16;
static_assert(kJoinWarps == kTileRows, "a warp a row");
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32, 2) k_kv_join(const __grid_constant__ KvAttnArgs a) {
  constexpr int E = D / 32;  // elements a lane
  __shared__ float so[kJoinWarps][D], sl[kJoinWarps], sm[kJoinWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int n_split = reinterpret_cast<const KvHeader*>(a.plan)->n_split;
  const int4* entry = reinterpret_cast<const int4*>(a.plan + a.L.split) + 2 * blockIdx.x;
  const int4 sp = entry[0], sq = entry[1];
  const int warp = (int)warp_id(), lane = (int)lane_id();
  const bool few = sp.y <= kJoinFew;
  const int head = (int)blockIdx.y, r = few ? warp : (int)blockIdx.z, rows = sq.z * a.G;
  if (!plan_filled(a.plan, a.L.sig) || (int)blockIdx.x >= n_split || (few ? blockIdx.z != 0 : r >= rows)) return;
  const int first = few ? 0 : warp, step = few ? 1 : kJoinWarps;
  const int64_t stride = (int64_t)a.nkv * kTileRows;
  const int64_t base = (int64_t)sp.x * stride + (int64_t)head * kTileRows + r;
  float m = -INFINITY, l = 0.0f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
  if (r < rows) {
    for (int i0 = first; i0 < sp.y; i0 += kJoinFlight * step) {
      float w[kJoinFlight], x[kJoinFlight][E];
#pragma unroll
      for (int k = 0; k < kJoinFlight; ++k) {
        const int i = i0 + k * step;
        w[k] = -INFINITY;
#pragma unroll
        for (int e = 0; e < E; ++e) x[k][e] = 0.0f;
        if (i < sp.y) {
          w[k] = a.part_l[base + i * stride];
          const float* src = a.part_o + (base + i * stride) * D + lane * E;
          if (E == 4) {
            const float4 f = *reinterpret_cast<const float4*>(src);
            x[k][0] = f.x;
            x[k][1] = f.y;
            x[k][E - 2] = f.z;
            x[k][E - 1] = f.w;
          } else {
            const float2 f = *reinterpret_cast<const float2*>(src);
            x[k][0] = f.x;
            x[k][1] = f.y;
          }
        }
      }
      float nm = m;
#pragma unroll
      for (int k = 0; k < kJoinFlight; ++k) nm = fmaxf(nm, w[k]);
      const float ref = nm == -INFINITY ? 0.0f : nm, c = m == -INFINITY ? 0.0f : ex2(m - ref);
      m = nm;
      l *= c;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= c;
#pragma unroll
      for (int k = 0; k < kJoinFlight; ++k) {
        const float wt = ex2(w[k] - ref);
        l += wt;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += wt * x[k][e];
      }
    }
  }
  if (!few) {
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
    if (lane == 0) {
      sl[warp] = l;
      sm[warp] = m;
    }
    __syncthreads();
    if (warp) return;
    m = -INFINITY;
    for (int i = 0; i < kJoinWarps; ++i) m = fmaxf(m, sm[i]);
    const float ref = m == -INFINITY ? 0.0f : m;
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    for (int i = 0; i < kJoinWarps; ++i) {
      const float c = sm[i] == -INFINITY ? 0.0f : ex2(sm[i] - ref);
      l += sl[i] * c;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += so[i][lane * E + e] * c;
    }
  }
  if (r >= rows) return;
  const bool none = l == 0.0f;
  const int i = r / a.G, h = head * a.G + r - i * a.G;
  uint16_t* dst = a.o + (int64_t)(sq.y + i) * a.so + h * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = none ? 0u : pack_bf16x2(__fdiv_rn(acc[e], l), __fdiv_rn(acc[e + 1], l));
  if (a.lse && lane == 0) a.lse[(int64_t)h * a.T + sq.y + i] = none ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Where the partial results lie in the workspace: the decode kernel's sums behind
// its rows, the chunk kernel's behind both.
struct KvWork {
  size_t part_l, chunk, bytes;
};
KvWork kv_work(const KvShape& s, const KvLayout& L) {
  // a cut tile's pieces lie in slots unit + index of the tile: below 2 max_units
  const size_t rows = L.max_tiles > 0 ? (size_t)(2 * L.max_units) * s.nkv * kTileRows : 0;
  KvWork w;
  w.part_l = rows * s.hd * 4;
  w.chunk = w.part_l + rows * 4;  // a multiple of 64
  w.bytes = w.chunk + kv_chunk_bytes(s) + 16;  // the chunk kernel stores 32 bytes at a time, the caller's is at 16
  return w;
}

template <int D, int NQ>
cudaError_t launch_decode(const KvAttnArgs& a, int64_t units, cudaStream_t st) {
  constexpr uint32_t bytes = DecodeSmem<D>::BYTES;
  const cudaError_t e = allow_smem<k_kv_decode<D, NQ>>((int)bytes);
  if (e != cudaSuccess) return e;
  note_launch();
  const int64_t warps = units * a.nkv;
  return launch_pdl(k_kv_decode<D, NQ>, dim3((unsigned)((warps + kDecodeWarps - 1) / kDecodeWarps)),
                    dim3(kDecodeWarps * 32), bytes, st, a);
}

}  // namespace
}  // namespace ws

using namespace ws;

extern "C" {

ws_status ws_attention_kv_workspace_size(const ws_kv_plan* plan, size_t* bytes) {
  KvShape s;
  const ws_status st = kv_shape(plan, &s);
  if (st != WS_OK) return st;
  if (!bytes) return WS_ERR_INVALID;
  *bytes = kv_work(s, kv_layout(s)).bytes;
  return WS_OK;
}

ws_status ws_attention_kv(const ws_kv_cache* cache, const ws_kv_plan* plan, const uint16_t* q,
                          int64_t q_stride, float scale, uint16_t* o, int64_t o_stride, float* lse,
                          void* workspace, size_t ws_bytes, ws_stream_t stream) {
  KvShape s;
  const ws_status c = kv_check(cache, plan, &s);
  if (c != WS_OK) return c;
  if (!q || !o || !workspace || !(scale > 0.0f) || !isfinite(scale)) return WS_ERR_INVALID;
  for (int64_t d : {q_stride, o_stride})
    if (d < (int64_t)s.nh * s.hd || d % 8 || d > (int64_t)1 << 31) return WS_ERR_SHAPE;
  for (const void* p : {(const void*)q, (const void*)o, (const void*)workspace})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return WS_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(lse) & 3u) return WS_ERR_ALIGN;
  KvAttnArgs a;
  a.L = kv_layout(s);
  const KvWork w = kv_work(s, a.L);
  if (ws_bytes < w.bytes) return WS_ERR_OOM;
  a.k = cache->k;
  a.v = cache->v;
  a.scale = cache->scale;
  a.plan = static_cast<const uint8_t*>(plan->data);
  a.table = plan->page_table;
  a.q = q;
  a.o = o;
  a.lse = lse;
  uint8_t* work = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(workspace) + 31) & ~uintptr_t(31));
  a.part_o = reinterpret_cast<float*>(work);
  a.part_l = reinterpret_cast<float*>(work + w.part_l);
  a.n_pages = cache->n_pages;
  a.sq = q_stride;
  a.so = o_stride;
  a.T = s.T;
  a.nkv = s.nkv;
  a.G = s.nh / s.nkv;
  a.max_pages = s.max_pages;
  a.sl2 = scale * kLog2e;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (a.L.c_max_tiles > 0) e = run_kv_chunk(a, s, work + w.chunk, st);
  if (e != cudaSuccess) return WS_ERR_CUDA;
  if (a.L.max_tiles > 0) {
    const bool few = std::min<int64_t>((int64_t)s.max_new * a.G, kTileRows) <= 8;  // rows of a tile
    if (s.hd == 64)
      e = few ? launch_decode<64, 1>(a, a.L.max_units, st) : launch_decode<64, 2>(a, a.L.max_units, st);
    else
      e = few ? launch_decode<128, 1>(a, a.L.max_units, st) : launch_decode<128, 2>(a, a.L.max_units, st);
    if (e != cudaSuccess) return WS_ERR_CUDA;
    // cut tiles: one share's end each at most
    const dim3 grid((unsigned)std::min<int64_t>(a.L.max_units, a.L.max_tiles), (unsigned)s.nkv,
                    (unsigned)std::min<int64_t>(kTileRows, (int64_t)s.max_new * a.G));
    note_launch();
    e = launch_pdl(s.hd == 64 ? k_kv_join<64> : k_kv_join<128>, grid, dim3(kJoinWarps * 32), 0, st, a);
  }
  return e == cudaSuccess ? WS_OK : WS_ERR_CUDA;
}

}  // extern "C"
