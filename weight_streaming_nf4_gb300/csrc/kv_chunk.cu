// kv_chunk.cu -- attention over the paged 8-bit cache for sequences of more
// than 16 rows (prompts, in chunks behind what the cache holds): the definition
// is that of kv_attention.cu, the products are tcgen05's.
//
// A tile is 256 rows (new token, head of the group) of one kv head, two slots of
// 128; a step is two pages.  For each step and slot
//   S = Q K^T    kind::f8f6f4: the key codes as TMA brings them, nothing decoded.
//                A row of Q enters as a power of two times hi + lo, hi in e4m3 and
//                lo in e5m2 (hi leaves at most eight of bf16's last places, either
//                way, so three bits hold them, at e5m2's range): exact down to 2^-14
//                of the row's largest element, off by 2^-21.8 of it below; two
//                products at twice fp16's rate cost what one fp16 product does
//   P = 2^(S c - m) as fp16 and, for every 16 tokens behind it, what fp16 leaves of it
//                (2^-22 of P for 2^-11), in the same columns of tensor memory
//   O += P V     kind::f16, two products, A from tensor memory, V decoded to fp16
//                (exact) by two warps, once for both slots
// A row is a thread's, so its maximum and sum need no exchange.  m moves only
// when a row's maximum has grown by 2^8 or more, as far as fp16 holds P (that the
// maximum may lag, and that two tiles of queries take turns on the tensor cores,
// are known from published attention algorithms; Shah et al., 2024, for the latter):
// then the softmax warps wait for the products before and rescale O in tensor
// memory.  Keys' scales go into c, values' into P (page_ref in kv_plan.cuh, as lazy
// as m).
// A tile of up to 128 rows has both slots on the same rows, on steps of their
// own (even, odd), joined at the end: without that the products would wait for
// the softmax at every step.
//
// Two prompts, 1800 + 1519 rows of 40 + 8 heads behind 6000 and 3392 tokens, take
// 413 us (0.93 PFLOP/s of the definition's products, three of which are made for
// two; the tensor pipe is busy 0.66 of the time).  A step takes some 4200 clocks
// where its products are 3.1 thousand: it is the chain of a slot's step, S to softmax to
// P V to the next S, over barriers, with the two slots' chains beside each other; a
// third does not fit in tensor memory at D = 128.  P's second part takes a quarter
// (without its products 0.88 of the time, without making it 0.96).  With P in one
// part, 3300 clocks for 2048, neither fewer products (an eighth of them: 0.88),
// nor a softmax without exponentials (0.99), nor values that are not decoded (1.0)
// shortened it much; halves of S as products of their own (N = 64) took 1.15, two
// warps that issue or a turn taken by the slots were no faster.  The rest is what a
// tile's beginning costs (queries staged, O written: some five steps).  With 14 + 2
// heads of 64 the two prompts take 136 us, 0.49 PFLOP/s: half the products on the
// same chain, the tensor pipe busy 0.36 of the time.
// Shares of equal cost, over all heads, one CTA an SM: a share that begins or
// ends inside a tile leaves a partial result, joined by k_kv_chunk_join in the
// order of the shares.
//
// Warps: 0 loads, 1 issues the products, 2 and 3 decode values, 4-7 and 8-11 are the
// slots' rows (three warps on each quarter of an SM: 168 registers a thread).  Every wait is bounded, by
// kWaitLimitNs of common.cuh.
#define WS_KV_TU 1
#include <math.h>

#include "kv_plan.cuh"

namespace ws {

cudaError_t kv_chunk_read_and_clear_dev_error(uint32_t* flags) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_dev_error, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_dev_error, &zero, sizeof(uint32_t));
}

namespace {

constexpr int kChThreads = 384;
constexpr int kSlotRows = 128;
constexpr int kStepTokens = 2 * kPage;
constexpr int kInfo = 64;      // pages of a window of the pages' list
constexpr int kLag = 8;        // powers of two by which a row's maximum may outgrow m
constexpr int kChMargin = 7;   // P 2^7: up to 2^15 in fp16

struct ChunkArgs {
  KvAttnArgs a;
  CUtensorMap tk;  // keys as [n_pages n_kv_heads][64][D] bytes
  float* part_o;   // [slot][kChunkRows][D], divided by their sums
  float* part_l;   // [slot][kChunkRows] log2 of their sums
};

template <int D>
struct ChSmem {
  static constexpr int KST = 3;  // steps of keys in flight
  static constexpr int RST = 2;  // of value codes
  static constexpr int VST = 2;  // decoded (two: the products' warp counts on it)
  static constexpr uint32_t QP = kSlotRows * D;          // one part of a slot's rows
  static constexpr uint32_t K = kStepTokens * D;
  static constexpr uint32_t V = kStepTokens * D * 2;
  static constexpr uint32_t OFF_K = 4 * QP;
  static constexpr uint32_t OFF_R = OFF_K + KST * K;
  static constexpr uint32_t OFF_V = OFF_R + RST * K;
  static constexpr uint32_t OFF_INFO = OFF_V + VST * V;
  static constexpr uint32_t OFF_ML = OFF_INFO + 2 * kInfo * 16;
  static constexpr uint32_t OFF_BAR = OFF_ML + kSlotRows * 16;
  static constexpr uint32_t BYTES = OFF_BAR + 512 + 1024;
};

// A page of a step: its place (-1: none) and scales.
struct PageInfo {
  int page;
  float ks, vs;
  int pad;
};

// A share's stretch of one (head, tile).
struct Seg {
  int head, tile, r0, rows;  // rows of the tile
  int seq, past, row0, n;
  int s0, s1;                // its steps of the tile's
  int slot;                  // of its partial result, -1: the tile is whole
  bool dual;                 // both slots on the same rows
};

struct Share {
  const int4 *tiles, *seqs, *units;
  int64_t begin, end, at;
  int W, u, tile, head, nkv, G;
  WS_DEVINL Share(const ChunkArgs& c, int unit, bool run) {
    const KvHeader* h = reinterpret_cast<const KvHeader*>(c.a.plan);
    tiles = reinterpret_cast<const int4*>(c.a.plan + c.a.L.c_tile);
    seqs = reinterpret_cast<const int4*>(c.a.plan + c.a.L.seq);
    units = reinterpret_cast<const int4*>(c.a.plan + c.a.L.c_unit);
    u = unit;
    nkv = c.a.nkv;
    G = c.a.G;
    W = h->c_steps;
    const int U = h->c_units;
    begin = end = at = 0;
    if (!run || u >= U) return;
    const int4 b = units[u], e = units[u + 1];
    tile = b.x;
    head = b.y;
    begin = at = (int64_t)head * W + tiles[tile].z + b.w;
    end = (int64_t)e.y * W + tiles[e.x].z + e.w;
  }
  WS_DEVINL bool next(Seg& s) {
    if (at >= end) return false;
    if (at != begin && (int64_t)(head + 1) * W == at) {  // the next head begins
      ++head;
      tile = 0;
    } else if (at != begin) {
      ++tile;
    }
    const int4 t = tiles[tile], q = seqs[t.x];
    const int64_t base = (int64_t)head * W + t.z;
    const int steps = tiles[tile + 1].z - t.z;
    s.head = head;
    s.tile = tile;
    s.seq = t.x;
    s.r0 = t.y;
    s.past = q.x;
    s.row0 = q.y;
    s.n = q.z;
    s.rows = min(kChunkRows, q.z * G - t.y);
    s.s0 = (int)(at - base);
    s.s1 = (int)min((int64_t)steps, end - base);
    s.dual = s.rows <= kSlotRows;
    // cut by this share's begin, or by its end
    s.slot = s.s0 > 0 ? u + units[u].z : s.s1 < steps ? u + units[u + 1].z : -1;
    at = base + s.s1;
    return true;
  }
};

WS_DEVINL void tc_mma_f8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A in tensor memory (fp16 pairs), B through a descriptor.
WS_DEVINL void tc_mma_f16_ta(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
WS_DEVINL void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
      "%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
WS_DEVINL void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Operand of D-byte rows, K-major, swizzled over D = 128 or 64 bytes; `base` is
// that of the 32 bytes of the contraction step.
template <int D>
WS_DEVINL uint64_t desc_bytes(uint32_t base) {
  if (D == 128) return smem_desc_sw128(base, 16, 1024);
  return (uint64_t)((base >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(512 >> 4) << 32) | (1ull << 46) |
         (4ull << 61);
}
// Where 16-byte piece c of row r lies in it.
template <int D>
WS_DEVINL uint32_t swizzled(int r, int c) {
  return D == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}
// True in one lane of a converged warp.
WS_DEVINL bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(p));
  return p != 0u;
}
// A wait: a poll, a vote and a branch where the barrier is through (mbar_wait's
// clock reading and the abort flag at every wait cost more than the products they
// wait for).  Every lane sees the phase complete for itself, since a vote orders
// no memory.  After 256 polls, and every 256 from then on, the clock and the other
// roles are looked at: kWaitLimitNs later, or where a role gave up, so does this one.
// The answer is the warp's.
struct WaitLimit {
  uint64_t t0 = 0;
  WS_DEVINL bool over(const volatile uint32_t* abort_flag) {
    const uint64_t now = globaltimer();
    if (t0 == 0) t0 = now;
    return *abort_flag != 0u || now - t0 > kWaitLimitNs;
  }
};
WS_DEVINL bool poll(uint64_t* bar, uint32_t parity, const volatile uint32_t* abort_flag) {
  WaitLimit limit;
  for (uint32_t it = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++it)
    if ((it & 255u) == 0u && __any_sync(0xffffffffu, limit.over(abort_flag))) return false;
  return true;
}
// The same for one thread.
WS_DEVINL bool poll_one(uint64_t* bar, uint32_t parity, const volatile uint32_t* abort_flag) {
  WaitLimit limit;
  for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it)
    if ((it & 255u) == 0u && limit.over(abort_flag)) return false;
  return true;
}
WS_DEVINL bool warp_all(bool v) { return __all_sync(0xffffffffu, v); }

// Two fp32 operations an instruction.
typedef unsigned long long f32x2;
WS_DEVINL f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
WS_DEVINL void unpair(f32x2 x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
WS_DEVINL f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
WS_DEVINL f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 32 of a row's scores as 2^(x cf - shift), as they lie in tensor memory: for every 16 tokens eight columns of fp16
// pairs and eight of what those leave.  Their sums are added to sum.
WS_DEVINL void weigh_plain(const uint32_t (&x)[32], f32x2 c2, f32x2 r2, f32x2 (&sum)[2], uint32_t (&p)[32]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float y0, y1;
    unpair(fma2(pair(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2, r2), y0, y1);
    y0 = ex2(y0);
    y1 = ex2(y1);
    sum[i & 1] = add2(sum[i & 1], pair(y0, y1));
    const int at = (i & 8) * 2 + (i & 7);
    split_f16x2(y0, y1, p[at], p[at + 8]);
  }
}
template <int D>
__global__ void __launch_bounds__(kChThreads, 1) k_kv_chunk(const __grid_constant__ ChunkArgs c) {
  using L = ChSmem<D>;
  constexpr int KST = L::KST, RST = L::RST, VST = L::VST;
  constexpr uint32_t TM_S = 0, TM_O = 2 * kStepTokens, TM_COLS = 512;
  constexpr uint32_t idS = (1u << 4) | ((kStepTokens >> 3) << 17) | ((kSlotRows >> 4) << 24);  // e4m3, e4m3, fp32
  constexpr uint32_t idLo = idS | (1u << 7);                                                   // e5m2, e4m3, fp32
  constexpr uint32_t idO = (1u << 4) | ((D >> 3) << 17) | ((kSlotRows >> 4) << 24);            // fp16, fp16, fp32
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = smem;  // [slot][hi, lo]
  uint8_t* sk = smem + L::OFF_K;
  uint8_t* sr = smem + L::OFF_R;
  uint8_t* sv = smem + L::OFF_V;
  PageInfo* info = reinterpret_cast<PageInfo*>(smem + L::OFF_INFO);  // [2][kInfo]
  float4* ml = reinterpret_cast<float4*>(smem + L::OFF_ML);          // slot 1's m, l, oref of each row
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* k_full = bars;
  uint64_t* k_empty = k_full + KST;
  uint64_t* r_full = k_empty + KST;
  uint64_t* r_empty = r_full + RST;
  uint64_t* v_full = r_empty + RST;
  uint64_t* v_empty = v_full + VST;
  uint64_t* q_full = v_empty + VST;      // [slot]
  uint64_t* s_full = q_full + 2;         // [slot]
  uint64_t* p_full = s_full + 2;         // [slot][half]
  uint64_t* o_done = p_full + 4;         // [slot][half]
  uint64_t* i_full = o_done + 4;         // [window]
  uint64_t* i_empty = i_full + 2;
  uint64_t* ml_full = i_empty + 2;
  uint64_t* o1_free = ml_full + 1;
  uint64_t* drain = o1_free + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  volatile uint32_t* skip_flag = tmem_slot + 2;

  const int warp = __shfl_sync(0xffffffffu, (int)warp_id(), 0), lane = (int)lane_id();
  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    *skip_flag = (*(volatile uint32_t*)&g_dev_error != 0u) ? 1u : 0u;
    for (int i = 0; i < KST; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < RST; ++i) {
      mbar_init(&r_full[i], 1);
      mbar_init(&r_empty[i], 2);
    }
    for (int i = 0; i < VST; ++i) {
      mbar_init(&v_full[i], 2);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], 4);
      mbar_init(&p_full[2 * i + 1], 4);
      mbar_init(&o_done[2 * i], 1);
      mbar_init(&o_done[2 * i + 1], 1);
      mbar_init(&i_full[i], 1);
      mbar_init(&i_empty[i], 10);
    }
    mbar_init(ml_full, 4);
    mbar_init(o1_free, 4);
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();
  const bool run = *skip_flag == 0u && plan_filled_or_say(c.a.plan, c.a.L.sig);
  Share share(c, (int)blockIdx.x, run);
  const KvAttnArgs& a = c.a;
  Seg sg = {};
  // Steps are numbered through the share; step n's pages are 2 n and 2 n + 1 of
  // the share's list of pages, in windows of kInfo.
  auto info_of = [&](int n, int half) -> const PageInfo& {
    return info[(2 * n + half) & (2 * kInfo - 1)];
  };
  auto give_up = [&](uint32_t why) {
    if (*abort_flag == 0u) atomicOr(&g_dev_error, why);
    *abort_flag = 1u;
  };
  // Enter the window that step n begins, if it begins one.
  auto window = [&](int n) {
    if (n & (kInfo / 2 - 1)) return true;
    const int w = n / (kInfo / 2);
    return poll(&i_full[w & 1], (uint32_t)(w >> 1) & 1u, abort_flag);
  };
  // Leave the window that step n ends.
  auto leave = [&](int n) {
    if (((n + 1) & (kInfo / 2 - 1)) == 0 && lane == 0) mbar_arrive(&i_empty[(n / (kInfo / 2)) & 1]);
  };

  if (warp == 0) {
    if (run) {
      // the whole warp walks: every kInfo pages it looks up the next window
      const int total = (int)(share.end - share.begin);
      Share ahead = share;  // the walk of the page list
      Seg as;
      bool more = ahead.next(as);
      int as_step = more ? as.s0 : 0;
      int n = 0;  // steps loaded
      bool ok = true;
      while (n < total && ok) {
        const int w = n / (kInfo / 2);
        // the window's pages: lane i has pages 2 i, 2 i + 1 = step n + i
        ok = poll(&i_empty[w & 1], ((uint32_t)(w >> 1) & 1u) ^ 1u, abort_flag);
        if (!ok) break;
        // lane i has step n + i; a segment or two make up a window, and each page costs one trip for all lanes
        int seq = 0, head = 0, p = 0, pend = 0;  // pages from pend on are seen by no row of the tile
        for (int filled = 0; filled < kInfo / 2 && more;) {
          const int cnt = min(kInfo / 2 - filled, as.s1 - as_step);
          if (lane >= filled && lane < filled + cnt) {
            seq = as.seq;
            head = as.head;
            p = 2 * (as_step + lane - filled);
            pend = (as.past + (as.r0 + as.rows - 1) / a.G) / kPage + 1;
          }
          filled += cnt;
          as_step += cnt;
          if (as_step == as.s1) {
            more = ahead.next(as);
            as_step = as.s0;
          }
        }
        PageInfo mine[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mine[h].page = p + h < pend ? a.table[(int64_t)seq * a.max_pages + p + h] : -1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mine[h].ks = mine[h].vs = 0.0f;
          if (mine[h].page >= a.n_pages) mine[h].page = -1;
          if (mine[h].page >= 0) {
            mine[h].page = mine[h].page * a.nkv + head;
            const float2 s = *(reinterpret_cast<const float2*>(a.scale) + mine[h].page);
            mine[h].ks = s.x;
            mine[h].vs = s.y;
          }
          info[(2 * (n + lane) + h) & (2 * kInfo - 1)] = mine[h];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_full[w & 1]);
        const int stop = min(total, n + kInfo / 2);
        if (lane == 0) {
          for (; n < stop; ++n) {
            const PageInfo p0 = info_of(n, 0), p1 = info_of(n, 1);
            const uint32_t bytes = ((p0.page >= 0) + (p1.page >= 0)) * kPage * D;
            const int ks = n % KST, rs = n % RST;
            if (!poll_one(&k_empty[ks], ((uint32_t)(n / KST) & 1u) ^ 1u, abort_flag)) break;
            mbar_arrive_expect_tx(&k_full[ks], bytes);
            uint8_t* dk = sk + ks * L::K;
            if (p0.page >= 0) tma_load_3d(dk, &c.tk, &k_full[ks], 0, 0, p0.page);
            if (p1.page >= 0) tma_load_3d(dk + kPage * D, &c.tk, &k_full[ks], 0, 0, p1.page);
            if (!poll_one(&r_empty[rs], ((uint32_t)(n / RST) & 1u) ^ 1u, abort_flag)) {
              mbar_wait(&k_full[ks], (uint32_t)(n / KST) & 1u, DERR_TIMEOUT_DRAIN);
              break;
            }
            mbar_arrive_expect_tx(&r_full[rs], bytes);
            uint8_t* dr = sr + rs * L::K;
            if (p0.page >= 0) bulk_load(dr, a.v + (int64_t)p0.page * (kPage * D), kPage * D, &r_full[rs]);
            if (p1.page >= 0)
              bulk_load(dr + kPage * D, a.v + (int64_t)p1.page * (kPage * D), kPage * D, &r_full[rs]);
          }
          if (n < stop) {
            give_up(DERR_TIMEOUT_EMPTY);
            ok = false;
          }
        }
        n = __shfl_sync(0xffffffffu, n, 0);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      // nothing may land after the CTA is gone
      if (lane == 0) {
        for (int i = max(0, n - KST); i < n; ++i)
          mbar_wait(&k_full[i % KST], (uint32_t)(i / KST) & 1u, DERR_TIMEOUT_DRAIN);
        for (int i = max(0, n - RST); i < n; ++i)
          mbar_wait(&r_full[i % RST], (uint32_t)(i / RST) & 1u, DERR_TIMEOUT_DRAIN);
      }
    }
  } else if (warp == 1) {
    // The whole warp walks, so that what the products take is in uniform
    // registers; one lane issues.
    if (run) {
      bool ok = true;
      uint32_t qn = 0, pn = 0;              // parities of each slot's segments and steps, a bit each
      int kst = 0, vst = 0;                 // stages in use, and their parities
      uint32_t kph = 0, vph = 0;
      auto wait = [&](uint64_t* b, uint32_t parity) {
        ok = poll(b, parity & 1u, abort_flag);
        return ok;
      };
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), base = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
      // descriptors: the low word moves, the high word stays
      const uint64_t dk0 = desc_bytes<D>(0u), dv0 = smem_desc_sw128(0u, 16, 1024);
      while (ok && share.next(sg)) {
        // Event e is step j of slot e & 1: both slots' of one step come together, or (dual) the steps in turn.
        // P V of event e, then S of event e + 2, the same slot's next.
        const int J = sg.s1 - sg.s0, E = sg.dual ? J : 2 * J;
#pragma unroll 1
        for (int e0 = -2; e0 < E && ok; e0 += 2) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int e = e0 + s;
            const bool begins = sg.dual || s == 0, ends = sg.dual || s == 1;  // the first, the last to use a step
            const bool pv = e >= 0 && e < E, next = e + 2 < E;
            // what is long there, before the slot's P
            if (pv && begins && !wait(&v_full[vst], vph)) break;
            if (next && begins && !wait(&k_full[kst], kph)) break;
            if (next && e < 0) {  // the slot's first of the segment
              if (!wait(&q_full[s], qn >> s)) break;
              qn ^= 1u << s;
            }
            if (pv) {
              const uint64_t v = dv0 + ((base + L::OFF_V + vst * L::V) >> 4);
              const uint32_t d = tm + TM_O + s * D, p = tm + TM_S + s * kStepTokens;
              if (!wait(&p_full[2 * s], pn >> s)) break;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int i = 0; i < kPage / 8; ++i)  // 16 tokens' P, then what fp16 leaves of it
                  tc_mma_f16_ta(d, p + i * 8, v + ((32 * (i >> 1)) >> 4), idO, (e < 2 && i == 0) ? 0u : 1u);
                tc_commit(&o_done[2 * s]);
              }
              __syncwarp();
              if (!wait(&p_full[2 * s + 1], pn >> s)) break;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int i = 0; i < kPage / 8; ++i)
                  tc_mma_f16_ta(d, p + kPage + i * 8, v + ((D * 128 + 32 * (i >> 1)) >> 4), idO, 1u);
                tc_commit(&o_done[2 * s + 1]);
                if (ends) tc_commit(&v_empty[vst]);
              }
              __syncwarp();
              pn ^= 1u << s;
              if (ends) {
                vst ^= 1;
                vph ^= vst == 0;
              }
            }
            if (next) {
              tc_fence_after();
              const uint64_t q = dk0 + ((base + s * 2 * L::QP) >> 4), k = dk0 + ((base + L::OFF_K + kst * L::K) >> 4);
              const uint32_t d = tm + TM_S + s * kStepTokens;
              if (elect_one()) {
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                  for (int i = 0; i < D / 32; ++i)
                    tc_mma_f8(d, q + ((part * L::QP + 32 * i) >> 4), k + ((32 * i) >> 4), part ? idLo : idS,
                              (part | i) ? 1u : 0u);
                tc_commit(&s_full[s]);
                if (ends) tc_commit(&k_empty[kst]);
              }
              __syncwarp();
              if (ends) {
                kst = kst == KST - 1 ? 0 : kst + 1;
                kph ^= kst == 0;
              }
            }
          }
        }
      }
      if (!ok) give_up(DERR_TIMEOUT_BFULL);
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      mbar_wait(drain, 0u, DERR_TIMEOUT_DRAIN);
    }
  } else if (warp < 4) {
    // ---- values: codes [D][64 tokens] of each page -> fp16 operand rows of 64 tokens
    if (run) {
      const int w = warp - 2;
      int n = 0;
      bool ok = true;
      while (ok && share.next(sg)) {
        const int kv_end = sg.past + sg.n;
        for (int j = sg.s0; j < sg.s1 && ok; ++j, ++n) {
          const int rs = n % RST, st = n % VST;
          ok = window(n) && poll(&v_empty[st], ((uint32_t)(n / VST) & 1u) ^ 1u, abort_flag) &&
               poll(&r_full[rs], (uint32_t)(n / RST) & 1u, abort_flag);
          if (!ok) break;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const bool have = info_of(n, h).page >= 0;
            const int left = kv_end - (2 * j + h) * kPage;  // tokens of the page that are the sequence's
            const uint8_t* src = sr + rs * L::K + h * (kPage * D);
            uint8_t* dst = sv + st * L::V + h * (D * 128);
            const int r0 = w * (D / 2) + (lane >> 2), u = lane & 3;
            uint4 x[D / 16];
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
              x[i] = have ? *reinterpret_cast<const uint4*>(src + (r0 + 8 * i) * kPage + 16 * u) : make_uint4(0, 0, 0, 0);
            if (left < kPage) {  // places behind the last token hold anything, NaN too
              uint32_t keep[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int m = left - 16 * u - 4 * e;
                keep[e] = m >= 4 ? 0xffffffffu : m <= 0 ? 0u : (1u << (8 * m)) - 1u;
              }
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                x[i].x &= keep[0];
                x[i].y &= keep[1];
                x[i].z &= keep[2];
                x[i].w &= keep[3];
              }
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              uint32_t y[8];
              decode4(x[i].x, y[0], y[1]);
              decode4(x[i].y, y[2], y[3]);
              decode4(x[i].z, y[4], y[5]);
              decode4(x[i].w, y[6], y[7]);
              sts128(dst + swizzled<128>(r0 + 8 * i, 2 * u), y[0], y[1], y[2], y[3]);
              sts128(dst + swizzled<128>(r0 + 8 * i, 2 * u + 1), y[4], y[5], y[6], y[7]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&r_empty[rs]);
            mbar_arrive(&v_full[st]);
          }
          leave(n);
        }
      }
      if (!ok) give_up(DERR_TIMEOUT_BEMPTY);
    }
  } else if (run) {
    // ---- rows: thread <-> row r of slot s
    const int s = (warp - 4) >> 2, q4 = warp & 3, r = q4 * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
    const uint32_t t_s = trow + TM_S + s * kStepTokens, t_o = trow + TM_O + s * D;
    uint8_t* q_hi = sq + s * 2 * L::QP;
    int n0 = 0;
    uint32_t sn = 0;         // steps of this slot
    uint32_t dn = 0;         // dual segments with both slots in use
    bool ok = true;
    auto wait = [&](uint64_t* b, uint32_t parity) {
      ok = poll(b, parity & 1u, abort_flag);
      return ok;
    };
    // This thread's row of Q in its two parts (the products of the segment
    // before are through: they gave the last S).  Returns its factor of S.  Two
    // passes over the row, its maximum and its codes, in a rolled loop: code that
    // runs once a segment comes from far away, eight instructions in some 300 clocks.
    auto stage = [&](const Seg& g) {
      if (g.dual && s >= g.s1 - g.s0) return 0.0f;  // the slot has no step
      const int local = g.dual ? r : s * kSlotRows + r, R = g.r0 + local, tok = R / a.G;
      const bool valid = local < g.rows;
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t)(g.row0 + (valid ? tok : 0)) * a.sq +
                                                        (g.head * a.G + (valid ? R - tok * a.G : 0)) * D);
      uint32_t top = 0;
#pragma unroll 1
      for (int i0 = 0; i0 < D / 8; i0 += 8) {
        uint4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = valid ? src[i0 + k] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          top = __vmaxu2(top, __vmaxu2(x[k].x & 0x7fff7fffu, x[k].y & 0x7fff7fffu));
          top = __vmaxu2(top, __vmaxu2(x[k].z & 0x7fff7fffu, x[k].w & 0x7fff7fffu));
          *reinterpret_cast<uint4*>(q_hi + (k & 1) * L::QP + swizzled<D>(r, (i0 + k) >> 1)) = x[k];
        }
      }
      top = max(top & 0xffffu, top >> 16);
      // the largest at (224, 448]; a row that is not finite gives NaN
      const int e = max((int)(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u), -126);
      const float qk = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 1
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t at = swizzled<D>(r, i);
        const uint4 n0 = *reinterpret_cast<const uint4*>(q_hi + at), n1 = *reinterpret_cast<const uint4*>(q_hi + L::QP + at);
        const uint32_t w[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
        uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float f0 = bf16_lo(w[k]) * qk, f1 = bf16_hi(w[k]) * qk;
          float g0, g1;
          const uint32_t ph = e4m3x2(f0, f1);
          e4m3x2_values(ph, g0, g1);
          hi[k >> 1] |= ph << (16 * (k & 1));
          lo[k >> 1] |= e5m2x2(f0 - g0, f1 - g1) << (16 * (k & 1));
        }
        *reinterpret_cast<uint4*>(q_hi + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(q_hi + L::QP + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[s]);
      return top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : a.sl2 * __uint_as_float((uint32_t)(e + 127) << 23);
    };
    bool have = false;  // a segment whose result is in O
    float qs = 0.0f, m = 0.0f, l = 0.0f, oref = 0.0f;  // oref: of O, see page_ref
    for (;;) {
      // the next segment's rows go first: its first products run beside the epilogue of the one before
      Seg nx;
      const bool more = share.next(nx);
      const float qn = more ? stage(nx) : 0.0f;
      const int J = sg.s1 - sg.s0;
      const int local = sg.dual ? r : s * kSlotRows + r;  // row of the tile
      if (have) {
        const bool active = !sg.dual || s < J, joined = sg.dual && J > 1;
        if (active && !wait(&o_done[2 * s + 1], sn - 1)) break;
        tc_fence_after();
        float m1 = -INFINITY, l1 = 0.0f, r1 = 0.0f;
        if (joined) {
          if (s == 1) {
            ml[r] = make_float4(m, l, oref, 0.0f);
            tc_fence_before();
          }
          __syncwarp();
          if (s == 1 && lane == 0) mbar_arrive(ml_full);
          // slot 0 takes both; slot 1 goes on when O of it has been read
          if (!wait(s == 1 ? o1_free : ml_full, dn)) break;
          ++dn;
          tc_fence_after();
          if (s == 0) {
            const float4 y = ml[r];
            m1 = y.x;
            l1 = y.y;
            r1 = y.z;
          }
        }
        if (!(sg.dual && s == 1)) {
          const bool valid = local < sg.rows;
          const int R = sg.r0 + local, tok = valid ? R / a.G : 0, h = sg.head * a.G + R - tok * a.G;
          const float mm = fmaxf(m, m1), ref = mm == -INFINITY ? 0.0f : mm;
          const float e0 = m == -INFINITY ? 0.0f : ex2(m - ref), e1 = m1 == -INFINITY ? 0.0f : ex2(m1 - ref);
          const float sum = l * e0 + l1 * e1;
          const bool none = sum == 0.0f;
          const float inv = none ? 0.0f : (1.0f / (1 << kChMargin)) / sum;
          const float f0 = e0 * inv, f1 = e1 * inv, g0 = pow2(oref), g1 = pow2(r1);
          const float lse2 = none ? -INFINITY : mm + log2f(sum);
          uint16_t* dst = a.o + (int64_t)(sg.row0 + tok) * a.so + h * D;
          const int64_t part = (int64_t)sg.slot * kChunkRows + local;
          const bool v8 = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0u && (a.so & 15) == 0;
#pragma unroll 1
          for (int cc = 0; cc < D; cc += 16) {
            uint32_t o0[16], o1[16];
            tmem_ld_32x32b_x16(t_o + cc, o0);
            if (joined) tmem_ld_32x32b_x16(trow + TM_O + D + cc, o1);
            tmem_ld_wait();
            if (valid) {
              float y[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                y[i] = none ? 0.0f : __uint_as_float(o0[i]) * f0 * g0;
                if (joined && !none) y[i] += __uint_as_float(o1[i]) * f1 * g1;
              }
              if (sg.slot >= 0) {
                float* d = c.part_o + part * D + cc;
#pragma unroll
                for (int i = 0; i < 16; i += 8)
                  st_global_v8(d + i, __float_as_uint(y[i]), __float_as_uint(y[i + 1]), __float_as_uint(y[i + 2]),
                               __float_as_uint(y[i + 3]), __float_as_uint(y[i + 4]), __float_as_uint(y[i + 5]),
                               __float_as_uint(y[i + 6]), __float_as_uint(y[i + 7]));
              } else {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
                if (v8) {
                  st_global_v8(dst + cc, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
                } else {
                  *reinterpret_cast<uint4*>(dst + cc) = make_uint4(w[0], w[1], w[2], w[3]);
                  *reinterpret_cast<uint4*>(dst + cc + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                }
              }
            }
            __syncwarp();
          }
          if (valid) {
            if (sg.slot >= 0)
              c.part_l[part] = lse2;
            else if (a.lse)
              a.lse[(int64_t)h * a.T + sg.row0 + tok] = lse2 * kLn2;
          }
          tc_fence_before();
          __syncwarp();
          if (joined && lane == 0) mbar_arrive(o1_free);
        }
      }
      if (!more) break;
      sg = nx;
      qs = qn;
      have = true;
      m = oref = -INFINITY;
      l = 0.0f;
      const int J1 = sg.s1 - sg.s0, mine = sg.dual ? r : s * kSlotRows + r;
      // tokens that the row sees; a row that is none (zero queries, nothing is stored) goes along with the last
      const int lim = mine < sg.rows ? sg.past + (sg.r0 + mine) / a.G + 1 : sg.past + sg.n;
      bool begun = false;  // something is in O
      for (int j = 0; j < J1; ++j) {
        const int n = n0 + j;
        if (!(ok = window(n))) break;
        if (sg.dual && (j & 1) != s) {
          leave(n);
          continue;
        }
        if (!wait(&s_full[s], sn)) break;
        tc_fence_after();
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const PageInfo pi = info_of(n, half);
          const uint32_t t_v = t_s + half * kPage;  // the page's scores, and in their place P
          float cf = qs * pi.ks;
          cf = cf < 1e-37f ? 1e-37f : cf;  // not below fp32's range: -inf * 0 is NaN
          const int vis = pi.page >= 0 ? lim - (2 * (sg.s0 + j) + half) * kPage : 0;  // of the page, seen
          // The ordinary page: all rows see all of it, m and O's reference stand and the scale of its P is a power of
          // two, 2^e, which goes into the exponent.  The sum bounds the largest: within fp16's range, and 2^(kLag + 1) of
          // m, both may stay.  (With 2^15 and 2^kLag as the limits, pages of scales that differ by 2 sent the two
          // prompts' rows the other way so often that they took 447 us for 416.)
          float vf;
          const float ve = scale_parts(pi.vs, vf), e = ve - oref + (float)kChMargin;
          const bool plain = vf == 1.0f && e >= -20.0f && e <= (float)(kChMargin + kLag) && vis >= kPage && m > -INFINITY;
          bool grown = false, rest = true;
          if (warp_all(plain)) {
            uint32_t p0[32], p1[32];
            uint32_t x0[32], x1[32];
            const float shift = m - e;
            const f32x2 c2 = pair(cf, cf), r2 = pair(-shift, -shift);
            f32x2 two[2] = {0ull, 0ull};  // two zeros each
            tmem_ld_32x32b_x32(t_v, x0);
            tmem_ld_wait();
            tmem_ld_32x32b_x32(t_v + 32, x1);
            weigh_plain(x0, c2, r2, two, p0);
            tmem_ld_wait();
            weigh_plain(x1, c2, r2, two, p1);
            float sum, other;
            unpair(add2(two[0], two[1]), sum, other);
            sum += other;
            grown = !(sum <= 65504.0f);
            sum *= pow2(-e);
            grown |= !(sum <= (float)(2 << kLag));
            rest = !warp_all(!grown);
            if (!rest) {
              l += sum;
              tmem_st_32x32b_x32(t_v, p0);
              tmem_st_32x32b_x32(t_v + 32, p1);
            }
          }
          if (rest) {
            // Any other page, 16 columns at a time: the maximum, then P in the place of S.
            float top = -INFINITY;
#pragma unroll 1
            for (int cc = 0; cc < kPage; cc += 16) {
              uint32_t x[16];
              tmem_ld_32x32b_x16(t_v + cc, x);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) top = cc + i < vis ? fmaxf(top, __uint_as_float(x[i])) : top;
            }
            top *= cf;
            const float lag = grown ? 0.0f : (float)kLag;
            const bool up = top > m + lag;
            const float nm = up ? top : m, need = page_ref(top - nm, ve);
            // (infinities of one sign give NaN, which the maximum passes over)
            const float nr = up || need > oref + lag ? fmaxf(floorf(oref + (m - nm)), need) : oref;
            if (__any_sync(0xffffffffu, up || nr != oref)) {
              const float f = up || nr != oref ? ex2((m - nm) + (oref - nr)) : 1.0f;
              if (up) l *= ex2(m - nm);
              m = nm;
              oref = nr;
              if (begun) {
                // O of the halves before
                if (!wait(&o_done[2 * s + (half ^ 1)], sn + half - 1)) break;
                tc_fence_after();
#pragma unroll 1
                for (int cc = 0; cc < D; cc += 16) {
                  uint32_t o[16];
                  tmem_ld_32x32b_x16(t_o + cc, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  tmem_st_32x32b_x16(t_o + cc, o);
                }
              }
            }
            const float ref = m == -INFINITY ? 0.0f : m;
            const float vr = page_factor(ve, oref, (float)kChMargin) * vf;
#pragma unroll 1
            for (int cc = 0; cc < kPage; cc += 16) {
              uint32_t x[16], p[16];
              tmem_ld_32x32b_x16(t_v + cc, x);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                // a row gets none of the scales of a page that it does not see, NaN included
                const bool in0 = cc + 2 * i < vis, in1 = cc + 2 * i + 1 < vis;
                const float y0 = in0 ? ex2(fmaf(__uint_as_float(x[2 * i]), cf, -ref)) : 0.0f;
                const float y1 = in1 ? ex2(fmaf(__uint_as_float(x[2 * i + 1]), cf, -ref)) : 0.0f;
                l += y0 + y1;
                split_f16x2(in0 ? y0 * vr : 0.0f, in1 ? y1 * vr : 0.0f, p[i], p[i + 8]);
              }
              tmem_st_32x32b_x16(t_v + cc, p);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * s + half]);
          begun = true;
        }
        if (!ok) break;
        ++sn;
        leave(n);
      }
      if (!ok) break;
      n0 += J1;
    }
    if (!ok) give_up(DERR_TIMEOUT_ACC);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, TM_COLS);
}

// Cut (head, tile) pairs: a row's pieces joined in the order of the shares, two
// rows a warp at a time, two pieces each in flight (the two prompts above: 413 us in
// all, with four rows a warp as long, with eight 425).
constexpr int kChJoinWarps = 8, kChJoinRows = 2;
template <int D>
__global__ void __launch_bounds__(kChJoinWarps * 32) k_kv_chunk_join(const __grid_constant__ ChunkArgs c) {
  constexpr int E = D / 32;
  pdl_wait();
  pdl_launch_dependents();
  const KvAttnArgs& a = c.a;
  const int n_split = reinterpret_cast<const KvHeader*>(a.plan)->c_split;
  const int4* entry = reinterpret_cast<const int4*>(a.plan + a.L.c_split) + 2 * blockIdx.x;
  const int4 sp = entry[0], sq = entry[1];
  const int lane = (int)lane_id(), rows = min(kChunkRows, sq.z * a.G - sp.z);
  const int first = ((int)blockIdx.y * kChJoinWarps + (int)warp_id()) * kChJoinRows;
  if (!plan_filled(a.plan, a.L.sig) || (int)blockIdx.x >= n_split || first >= rows) return;
  const int64_t base = (int64_t)sp.x * kChunkRows;
  float m[kChJoinRows], sum[kChJoinRows], acc[kChJoinRows][E];
#pragma unroll
  for (int r = 0; r < kChJoinRows; ++r) {
    m[r] = -INFINITY;
    sum[r] = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[r][e] = 0.0f;
  }
#pragma unroll 2
  for (int i = 0; i < sp.y; ++i) {
    float w[kChJoinRows], x[kChJoinRows][E];
#pragma unroll
    for (int r = 0; r < kChJoinRows; ++r) {
      const int64_t at = base + (int64_t)i * kChunkRows + min(first + r, rows - 1);
      w[r] = c.part_l[at];
      const float* src = c.part_o + at * D + lane * E;
      if (E == 4) {
        const float4 f = *reinterpret_cast<const float4*>(src);
        x[r][0] = f.x;
        x[r][1] = f.y;
        x[r][E - 2] = f.z;
        x[r][E - 1] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(src);
        x[r][0] = f.x;
        x[r][1] = f.y;
      }
    }
#pragma unroll
    for (int r = 0; r < kChJoinRows; ++r) {
      const float nm = fmaxf(m[r], w[r]), ref = nm == -INFINITY ? 0.0f : nm;
      const float old = m[r] == -INFINITY ? 0.0f : ex2(m[r] - ref), now = ex2(w[r] - ref);
      m[r] = nm;
      sum[r] = sum[r] * old + now;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[r][e] = acc[r][e] * old + now * x[r][e];
    }
  }
#pragma unroll
  for (int r = 0; r < kChJoinRows; ++r) {
    if (first + r >= rows) break;
    const bool none = sum[r] == 0.0f;
    const int R = sp.z + first + r, tok = R / a.G, h = sp.w * a.G + R - tok * a.G;
    uint16_t* dst = a.o + (int64_t)(sq.y + tok) * a.so + h * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) =
          none ? 0u : pack_bf16x2(__fdiv_rn(acc[r][e], sum[r]), __fdiv_rn(acc[r][e + 1], sum[r]));
    if (a.lse && lane == 0)
      a.lse[(int64_t)h * a.T + sq.y + tok] = none ? -INFINITY : (m[r] + log2f(sum[r])) * kLn2;
  }
}

template <int D>
cudaError_t launch_chunk(const ChunkArgs& c, cudaStream_t st) {
  const cudaError_t e = allow_smem<k_kv_chunk<D>>((int)ChSmem<D>::BYTES);
  if (e != cudaSuccess) return e;
  note_launch();
  const cudaError_t f = launch_pdl(k_kv_chunk<D>, dim3((unsigned)c.a.L.c_max_units), dim3(kChThreads),
                                   ChSmem<D>::BYTES, st, c);
  if (f != cudaSuccess) return f;
  note_launch();
  return launch_pdl(k_kv_chunk_join<D>, dim3((unsigned)c.a.L.c_max_units, kChunkRows / (kChJoinWarps * kChJoinRows)),
                    dim3(kChJoinWarps * 32), 0, st, c);
}

// Partial results lie in slots unit + index of the cut pair: below 2 units.
size_t chunk_rows() { return (size_t)2 * device_sm_count() * kChunkRows; }

}  // namespace

size_t kv_chunk_bytes(const KvShape& s) {
  return kv_chunk_tiles(s) > 0 ? chunk_rows() * ((size_t)s.hd + 1) * 4 : 0;
}

cudaError_t run_kv_chunk(const KvAttnArgs& a, const KvShape& s, void* partial, cudaStream_t st) {
  ChunkArgs c;
  c.a = a;
  if (!tmap_u8_pages(&c.tk, a.k, (uint32_t)s.hd, kPage, (uint64_t)a.n_pages * s.nkv)) return cudaErrorInvalidValue;
  c.part_o = static_cast<float*>(partial);
  c.part_l = c.part_o + chunk_rows() * s.hd;
  return s.hd == 64 ? launch_chunk<64>(c, st) : launch_chunk<128>(c, st);
}

}  // namespace ws
