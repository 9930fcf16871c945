// lora_few.cu -- the many-adapter NF4 linear for few rows: y = x W'^T + the
// adapter term, up to 64 rows at a time (decode), and the input gradient
// dX = dY W' + the adapter term, up to 64.
//
// Bound by decoding the codes (about 3.5 integer instructions a weight, on a
// pipe of 64 lanes an SM), then by reading them.  The dequant GEMM's tile has
// the activation rows as the 128-row operand and hands over 64-deep steps; with
// few rows its time is that handshake.  Here the WEIGHT rows are the 128-row
// operand and the rows of x the N-wide one (32 or 64), and a step is 256
// deep: sixteen warps decode 128 x 256 weights, each thread one 64-weight block
// (one value table for 64 weights), then hand over once; one thread loads x by
// TMA and one issues the tensor-core products (tcgen05, fp32 sums in tensor
// memory) of one step while the next is decoded.
//
// Forward: the weights go from registers into tensor memory, a row a lane, as
// the products' first operand (through shared memory a step takes as long).  The
// shared memory that is left holds the factors of the tile's rows (4 KB a row in
// bf16), brought by bulk copies while the tile's steps run; read from L2 in the
// epilogue, 48 rows of 48 adapters at 27648 x 5120 took 74 us, this way 66.  The
// input gradient wants the weights' columns as its rows: they go through shared
// memory, which keeps their orientation.
//
// Measured (weights from DRAM): 48 rows of 48 adapters at 27648 x 5120 take 66
// us with the kernel before it; a step takes 1.2 us, 0.93 of them the integer
// pipe's (counted: 224 instructions a thread).
//
// Schedule: the (tile, step) iterations of the whole problem are cut into equal
// contiguous ranges, one per CTA, all resident at once.  A tile cut by range
// ends is finished by the CTA that holds its first steps (its range's last
// piece): it adds the later CTAs' partial sums, which those make first of all,
// in step order.  So results depend on the shape and the SM count alone.
//
// Starts beside the kernel that makes U (programmatic launch): weights and x
// are read before the wait for it (that kernel has itself waited for everything
// earlier); U, the adapters, the workspace and y after.
#define WS_FEW_TU 1
#include "common.cuh"
#include "kernels.h"
#include "nf4_decode.cuh"

namespace ws {

cudaError_t few_read_and_clear_dev_error(uint32_t* flags) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_dev_error, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_dev_error, &zero, sizeof(uint32_t));
}

namespace {

constexpr int kDecWarps = 16, kDecThreads = kDecWarps * 32;
constexpr int kFewThreads = kDecThreads + 64;  // and a warp for the products, one for x
constexpr int kRows = 128;              // weight rows of a tile
constexpr uint32_t kABytes = 4 * 16384; // a step's operand: four 64-deep sub-tiles of 128 rows

template <int NX, bool BWD, bool F16>
struct Cfg {
  static constexpr uint32_t X_BYTES = NX * 512;  // a step of x: four sub-tiles of NX rows
  static constexpr int XS = NX == 64 ? 3 : 4;    // steps of x in flight
  // The adapters' factors of a tile (forward): slots of one row of x each, 16
  // values for each of 128 outputs; RP slots for each of the four groups of CPW
  // rows that share an epilogue warp.
  static constexpr int RP = F16 ? 8 : 4;
  static constexpr uint32_t ROW_BYTES = kRows * 16 * (F16 ? 2 : 4);
  static constexpr uint32_t OFF_A = 0, OFF_F = 0, OFF_X = BWD ? 2 * kABytes : 4 * RP * ROW_BYTES,
                            OFF_BAR = OFF_X + XS * X_BYTES;
  static constexpr uint32_t SMEM = OFF_BAR + 192 + 1024;  // + alignment slack
  static_assert(SMEM <= 227u * 1024u, "shared memory");
  // tensor memory: the sums, and in the forward two steps of weights (a row a
  // lane, two values a column)
  static constexpr uint32_t COL_A = 128, TMEM_COLS = BWD ? 4 * NX : 512;
  // input gradient: the products' sums in two buffers of NX columns, and after
  // them the running sums that they are added to (kGroup)
  static constexpr int NACC = BWD ? 2 : 1;
  static constexpr uint32_t COL_RUN = 2 * NX;
  static constexpr int CPW = NX / 4;             // accumulator columns (rows of x) of one epilogue warp
  static_assert(NX == 32 || NX == 64, "rows of x");
};

// D[tmem] (+)= A[tmem] * B[smem desc], kind::f16 (bf16 in, fp32 sums).
WS_DEVINL void tc_mma_f16_ta(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
WS_DEVINL float4 lds128f(uint32_t a) {
  float4 r;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
               : "r"(a)
               : "memory");
  return r;
}
// True in one lane of a converged warp.
WS_DEVINL bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(p));
  return p != 0u;
}
WS_DEVINL void tmem_ld_x4(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr)
               : "memory");
}

WS_DEVINL void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
WS_DEVINL void tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Steps (256 products each) of an fp32 gradient's sum that are left to the
// tensor cores, which cut off what their accumulator cannot hold: 28 of them
// were 6.9e-6 off (root mean square, N = 27648).  Even, as steps run in pairs.
constexpr int kGroup = 4;
static_assert(kGroup % 2 == 0, "take() sees each segment's first step");

// BWD: the input gradient.  The tile is 128 columns k of W', the contraction
// runs over its rows n, x is dY and y is dX; a thread decodes one 64-weight
// block of one row per step, 64 consecutive columns of the operand, which keeps
// W's own orientation (MN-major).  F is A [16, K], fp32.
template <int NX, bool BWD, bool F16>
__global__ void __launch_bounds__(kFewThreads, 1)
    k_few(const __grid_constant__ CUtensorMap tmX, const FewArgs a) {
  using C = Cfg<NX, BWD, F16>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [2] a step's weights are there
  uint64_t* empty = full + 2;                                       // [2] ... and have been used
  uint64_t* xfull = empty + 2;                                      // [XS] the same for x
  uint64_t* xempty = xfull + C::XS;
  uint64_t* acc_done = xempty + C::XS;                              // [NACC] a segment's sums are complete
  uint64_t* acc_free = acc_done + C::NACC;                          // [NACC] ... and have been read
  uint64_t* fac = acc_free + C::NACC;                               // factors have landed
  uint32_t* misc = reinterpret_cast<uint32_t*>(fac + 1);
  volatile uint32_t* abort_flag = misc + 1;
  volatile uint32_t* got_flag = misc + 2;
  // (the shuffle tells the compiler that a warp's index is one value)
  const int warp = __shfl_sync(0xffffffffu, (int)warp_id(), 0), lane = (int)lane_id();
  // this CTA's range: base iterations, one more for the first `extra` CTAs
  const int S = a.steps, u = (int)blockIdx.x;
  const int pb = u * a.base + min(u, a.extra), n_all = a.base + (u < a.extra ? 1 : 0);
  const int tile0 = (int)((uint32_t)pb / (uint32_t)S), step0 = pb - tile0 * S;

  // Codes of the thread's 64-weight block, two steps in registers and two more
  // on their way to L2; the first are asked for before anything is set up.
  // Forward: weight row r of the tile (a warp: the 32 lanes of tensor memory
  // that it may write), block t of the step.  BWD: weight row r of the step,
  // block t of the tile.
  const int r = (int)threadIdx.x & (BWD ? 255 : 127);
  const int t = (int)threadIdx.x >> (BWD ? 8 : 7);
  const int NO = BWD ? a.K : a.N;  // output columns
  struct Codes {
    uint4 w[2];
    float s;
  };
  const int64_t kb = a.K / 2;
  int lt = tile0, ls = step0, left = warp < kDecWarps ? n_all : 0;  // next step to load
  const uint8_t* cp = a.codes;
  const float* sp = a.absmax;
  auto seek = [&]() {
    if constexpr (BWD) {
      // blocks past the last column repeat it: their sums are not stored
      const int kblk = min(lt * 2 + t, a.K / 64 - 1);
      const int64_t n = (int64_t)ls * 256 + r;
      cp = a.codes + n * kb + kblk * 32;
      sp = a.absmax + (int64_t)kblk * a.N + n;
    } else {
      // rows past the last repeat it: their sums are not stored
      const int n = min(lt * kRows + r, a.N - 1);
      cp = a.codes + n * kb + (int64_t)ls * 128 + t * 32;
      sp = a.absmax + ((int64_t)ls * 4 + t) * a.N + n;
    }
  };
  const int64_t cp_step = BWD ? 256 * kb : 128, sp_step = BWD ? 256 : (int64_t)4 * a.N;
  // blocks of step s that exist: the last step may end inside it
  auto inside = [&](int s) { return BWD ? s * 256 + r < a.N : s * 256 + t * 64 < a.K; };
  auto load = [&](Codes& f) {
    if (left <= 0) return;
    // blocks past the end take codes that exist and a scale of 0
    const bool in = inside(ls);
    const uint4* c = reinterpret_cast<const uint4*>(in ? cp : a.codes);
    f.w[0] = __ldg(c);
    f.w[1] = __ldg(c + 1);
    f.s = in ? __ldg(sp) : 0.0f;
    if (left > 2 && ls + 2 < S && inside(ls + 2)) {
      asm volatile("prefetch.global.L2 [%0];" ::"l"(cp + 2 * cp_step));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(sp + 2 * sp_step));
    }
    --left;
    if (++ls == S) {
      ls = 0;
      ++lt;
      seek();
    } else {
      cp += cp_step;
      sp += sp_step;
    }
  };
  Codes f0{}, f1{};
  if (warp < kDecWarps) {
    seek();
    load(f0);
    load(f1);
  }
  if (threadIdx.x == 32) *abort_flag = *(volatile uint32_t*)&g_dev_error;  // an earlier kernel gave up: do nothing
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&full[s], kDecWarps);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < C::XS; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], 1);
    }
    for (int s = 0; s < C::NACC; ++s) {
      mbar_init(&acc_done[s], 1);
      mbar_init(&acc_free[s], kDecWarps);
    }
    mbar_init(fac, 1);
    fence_barrier_init();
  }
  if (warp == kDecWarps) {
    tmem_alloc(misc, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const bool skip = *abort_flag != 0u;
  const int n_it = skip ? 0 : n_all;
  // Steps of a segment: a piece is one, but that of an fp32 gradient kGroup
  // steps, after which its sums move to the running ones.
  const int group = BWD && a.out_f32 ? kGroup : 0x7fffffff;

  if (warp == kDecWarps) {
    // ------------------------------------------------------------ the products
    // The whole warp runs the loop and one lane issues: descriptors then stay
    // in uniform registers (issued from a single-lane branch, a step's sixteen
    // products took 2000 cycles to issue, as long as decoding it).
    const bool leader = elect_one();
    // (bit 15: the weights' operand is MN-major)
    constexpr uint32_t idesc = idesc_bf16_f32(kRows, NX, 0u) | (BWD ? 1u << 15 : 0u);
    // BWD: 8 rows n of a 64-column group make 1024 bytes, the two column groups
    // lie 1024 apart and 8-row groups 2048, so a 16-deep slice is 4096 bytes on.
    const uint64_t ad0 = smem_desc_sw128(smem_u32(smem + C::OFF_A), 1024, 2048);
    const uint64_t bd0 = smem_desc_sw128(smem_u32(smem + C::OFF_X), 16, 1024);
    int step = step0, xs = 0, in_seg = 0, b = 0;
    uint32_t xph = 0, fph = 1, last_ph = 0;  // phases of acc_free[b], and of the last acc_done
    int last_b = -1;
    bool first = true;  // of its segment
    for (int q = 0; q < n_it; ++q) {
      const int s = q & 1;
      bool ok = *abort_flag == 0u && mbar_wait(&full[s], (uint32_t)(q >> 1) & 1u, DERR_TIMEOUT_FULL) &&
                mbar_wait(&xfull[xs], xph, DERR_TIMEOUT_FULL) &&
                (!first || mbar_wait(&acc_free[b], fph, DERR_TIMEOUT_ACC));
      if (!__all_sync(0xffffffffu, ok)) {
        *abort_flag = 1u;
        break;
      }
      tc_fence_after();
      const bool tile_end = ++step == S;
      const bool end = tile_end || q + 1 == n_it || ++in_seg == group;
      if (leader) {
        const uint32_t acc = tmem + (uint32_t)(b * NX);
        const uint64_t ad = ad0 + (uint64_t)(s * (kABytes >> 4));
        const uint64_t bd = bd0 + (uint64_t)(xs * (C::X_BYTES >> 4));
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t xd = bd + (uint64_t)(t * NX * 8 + 2 * k);
            const uint32_t more = (t > 0 || k > 0 || !first) ? 1u : 0u;
            if constexpr (BWD) tc_mma_f16(acc, ad + (uint64_t)((t * 4 + k) * 256), xd, idesc, more);
            else tc_mma_f16_ta(acc, tmem + C::COL_A + (uint32_t)(s * 128 + (t * 4 + k) * 8), xd, idesc, more);
          }
        tc_commit(&empty[s]);
        tc_commit(&xempty[xs]);
        if (end) tc_commit(&acc_done[b]);
      }
      __syncwarp();
      if (++xs == C::XS) {
        xs = 0;
        xph ^= 1u;
      }
      first = end;
      if (tile_end) step = 0;
      if (end) {
        in_seg = 0;
        last_b = b;
        last_ph = fph ^ 1u;
        if (++b == C::NACC) {
          b = 0;
          fph ^= 1u;
        }
      }
    }
    // every product has completed before tensor memory is freed (the last
    // piece's commit covers all before it)
    if (last_b >= 0) mbar_wait(&acc_done[last_b], last_ph, DERR_TIMEOUT_DRAIN);
    if (*abort_flag) {
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 200000ull) __nanosleep(1000);
    }
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();
  } else if (warp == kDecWarps + 1) {
    // ------------------------------------------------------------ x
    if (lane == 0) {
      tma_prefetch_desc(&tmX);
      int step = step0, xs = 0;
      uint32_t ph = 1;
      for (int q = 0; q < n_it; ++q) {
        if (*abort_flag || !mbar_wait(&xempty[xs], ph, DERR_TIMEOUT_EMPTY)) {
          *abort_flag = 1u;
          break;
        }
        mbar_arrive_expect_tx(&xfull[xs], C::X_BYTES);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          tma_load_2d(smem + C::OFF_X + xs * C::X_BYTES + t * (NX * 128), &tmX, &xfull[xs], step * 256 + t * 64, 0);
        if (++xs == C::XS) {
          xs = 0;
          ph ^= 1u;
        }
        if (++step == S) step = 0;
      }
      if (*abort_flag) {  // copies in flight land first
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 200000ull) __nanosleep(1000);
      }
    }
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();
  } else {
    // ------------------------------------------------------------ decode and epilogue
    // BWD: the eight lanes of a quarter warp are eight rows, which the swizzle
    // keeps apart.
    uint32_t dst[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      dst[i] = smem_u32(smem + C::OFF_A) +
               (uint32_t)((r >> 3) * 2048 + t * 1024 + (r & 7) * 128 + ((i ^ (r & 7)) << 4));
    const uint32_t ta = tmem + ((uint32_t)(r & ~31) << 16) + C::COL_A + (uint32_t)t * 32;
    auto decode = [&](const Codes& f, int s) {
      const Nf4Table tb = make_table(f.s);
      const uint32_t w[8] = {f.w[0].x, f.w[0].y, f.w[0].z, f.w[0].w, f.w[1].x, f.w[1].y, f.w[1].z, f.w[1].w};
      if constexpr (BWD) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = dq8(w[i], tb);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst[i] + (uint32_t)s * kABytes), "r"(v.x),
                       "r"(v.y), "r"(v.z), "r"(v.w)
                       : "memory");
        }
        fence_proxy_async_smem();
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t v[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 d = dq8(w[4 * h + i], tb);
            v[4 * i] = d.x, v[4 * i + 1] = d.y, v[4 * i + 2] = d.z, v[4 * i + 3] = d.w;
          }
          tmem_st_32x32b_x16(ta + (uint32_t)(s * 128 + h * 16), v);
        }
        tmem_st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
    };
    bool waited = false;  // for the earlier kernels
    uint32_t seg = 0;     // segments read
    // The piece that ends with iteration q: tile `tile`, whether it holds the
    // tile's first and its last step.
    int q = 0;            // iterations made
    uint32_t fac_ph = 0;
    // One warp: the factors of the p-th RP rows of every group, for tile `tile`.
    // The plan and the adapters are older than the kernel before this one.
    auto ask = [&](int tile, int p) {
      if constexpr (!BWD) {
        constexpr int EB = F16 ? 2 : 4;
        const int n0 = tile * kRows, m = lane / C::RP * C::CPW + p * C::RP + lane % C::RP;
        const uint32_t bytes = (uint32_t)min(kRows, a.N - n0) * 16 * EB;
        const int ad = lane < 4 * C::RP && m < a.M ? a.row[m] : -1;
        const uint32_t some = __ballot_sync(0xffffffffu, ad >= 0);
        if (lane == 0) mbar_arrive_expect_tx(fac, (uint32_t)__popc(some) * bytes);
        __syncwarp();
        if (ad >= 0)
          bulk_load(smem + C::OFF_F + lane * C::ROW_BYTES,
                    static_cast<const uint8_t*>(a.F) + (ad * a.stride + (int64_t)n0 * 16) * EB, bytes, fac);
      }
    };
    // The next segment's sums, added to the running ones or (had = false) the
    // first of them.
    auto drain = [&](bool had) {
      const int b = (int)(seg % C::NACC);
      if (!*abort_flag && !mbar_wait(&acc_done[b], (seg / C::NACC) & 1u, DERR_TIMEOUT_ACC)) *abort_flag = 1u;
      tc_fence_after();
      __syncwarp();
      const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(warp / 4 * C::CPW);
#pragma unroll
      for (int c = 0; c < C::CPW; c += 8) {
        uint32_t v[8], run[8] = {};
        tmem_ld_x8(at + (uint32_t)(b * NX + c), v);
        if (had) tmem_ld_x8(at + C::COL_RUN + (uint32_t)c, run);
        tmem_ld_wait();
        if (had)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(__uint_as_float(run[e]) + __uint_as_float(v[e]));
        tmem_st_x8(at + C::COL_RUN + (uint32_t)c, v);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_free[b]);
      ++seg;
    };
    // had: the piece has running sums, the last segment's among them
    auto epilogue = [&](int tile, bool head, bool tail, bool had) {
      const int q4 = warp & 3, c0 = warp / 4 * C::CPW;  // lanes (weight rows) and columns of this warp
      const int nl = q4 * 32 + lane, n = tile * kRows + nl;
      int row_ad = -1;     // of the warp's rows, a lane each
      float row_sc = 0.0f;
      if (!BWD && head) {
        if (lane < C::CPW && c0 + lane < a.M) row_ad = a.row[c0 + lane];
        row_sc = a.scale[max(row_ad, 0)];
      }
      const int ab = (int)(seg % C::NACC);
      const bool ok = !*abort_flag && (had || mbar_wait(&acc_done[ab], (seg / C::NACC) & 1u, DERR_TIMEOUT_ACC));
      const uint32_t sums = !BWD ? 0u : had ? C::COL_RUN : (uint32_t)(ab * NX);  // column of the sums
      if (!had) ++seg;
      if (!ok) *abort_flag = 1u;
      tc_fence_after();
      if (!waited) {
        pdl_wait();
        pdl_launch_dependents();
        waited = true;
      }
      if (!BWD && head && lane < C::CPW / 2 && c0 + 2 * lane < a.M)  // P's rows, to L1
        asm volatile("prefetch.global.L1 [%0];" ::"l"(a.P + (int64_t)(c0 + 2 * lane) * 16));
      int last = u;  // CTA that holds the tile's last step
      if (head && !tail) {
        const int i = (tile + 1) * S - 1, cut = a.extra * (a.base + 1);
        last = i < cut ? i / (a.base + 1) : a.extra + (i - cut) / a.base;
        if (warp == 0) {  // a lane polls every 32nd flag
          bool got = ok;
          for (int v = u + 1 + lane; v <= last && got; v += 32)
            got = wait_flag_bounded(a.flags + v, 1u, kWaitLimitNs, DERR_TIMEOUT_PEER);
          got = __all_sync(0xffffffffu, got);
          __threadfence();
          if (lane == 0) *got_flag = got ? 1u : 0u;
        }
        named_bar_sync(1, kDecThreads);
        if (*got_flag == 0u) last = u;
      }
#pragma unroll(BWD ? 2 : 1)
      for (int cc = 0; cc < C::CPW; cc += 4) {
        uint32_t raw[4];
        tmem_ld_x4(tmem + ((uint32_t)(q4 * 32) << 16) + sums + (uint32_t)(c0 + cc), raw);
        tmem_ld_wait();
        if (cc + 4 == C::CPW && !had) {  // the sums are in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_free[ab]);
        }
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(raw[e]);
        if (!head) {  // a later piece of its tile: hand it over
          float* p = a.partial + (int64_t)(u * NX + c0 + cc) * kRows + nl;
#pragma unroll
          for (int e = 0; e < 4; ++e) __stcg(p + e * kRows, v[e]);
          continue;
        }
        // later pieces in step order, four at a time in flight
        for (int w = u + 1; w <= last; w += 4) {
          float x[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float* p = a.partial + (int64_t)((w + i) * NX + c0 + cc) * kRows + nl;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] = w + i <= last ? __ldcg(p + e * kRows) : 0.0f;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += x[i][e];
        }
        float d[4];
        if constexpr (BWD) {
          int ad[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) ad[e] = c0 + cc + e < a.M && n < NO ? a.row[c0 + cc + e] : -1;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            d[e] = -0.0f;  // changes no sum
            if (ad[e] < 0) continue;
            const float4* up = reinterpret_cast<const float4*>(a.P + (int64_t)(c0 + cc + e) * 16);
            const int64_t o = ad[e] * a.stride + n;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 x = up[j];
              float b[4];
              const float* f = static_cast<const float*>(a.F) + o + (int64_t)(4 * j) * a.K;
              b[0] = f[0], b[1] = f[a.K], b[2] = f[2 * (int64_t)a.K], b[3] = f[3 * (int64_t)a.K];
              d[e] = fmaf(x.x, b[0], d[e]), d[e] = fmaf(x.y, b[1], d[e]);
              d[e] = fmaf(x.z, b[2], d[e]), d[e] = fmaf(x.w, b[3], d[e]);
            }
            d[e] *= a.scale[ad[e]];
            if (a.mask) {
              const int64_t at = (int64_t)(c0 + cc + e) * a.K + n;
              if (!((a.mask[at >> 5] >> (at & 31)) & 1u)) d[e] = -0.0f;  // dropped here
            }
          }
        } else {
          if (cc % C::RP == 0) {
            if (!*abort_flag && !mbar_wait(fac, fac_ph, DERR_TIMEOUT_FULL)) *abort_flag = 1u;
            fac_ph ^= 1u;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            d[e] = 0.0f;
            const uint32_t f = smem_u32(smem + C::OFF_F) +
                               (uint32_t)(warp / 4 * C::RP + cc % C::RP + e) * C::ROW_BYTES + (uint32_t)nl * (F16 ? 32 : 64);
            const float4* up = reinterpret_cast<const float4*>(a.P + (int64_t)min(c0 + cc + e, a.M - 1) * 16);
            // the 16-byte parts in an order that sets eight lanes on eight
            // places of the banks
            if constexpr (F16) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int j = i ^ ((lane >> 2) & 1);
                const float4 w = lds128f(f + (uint32_t)j * 16), x = up[2 * j], z = up[2 * j + 1];
                d[e] = fmaf(x.x, bf16_lo(__float_as_uint(w.x)), d[e]), d[e] = fmaf(x.y, bf16_hi(__float_as_uint(w.x)), d[e]);
                d[e] = fmaf(x.z, bf16_lo(__float_as_uint(w.y)), d[e]), d[e] = fmaf(x.w, bf16_hi(__float_as_uint(w.y)), d[e]);
                d[e] = fmaf(z.x, bf16_lo(__float_as_uint(w.z)), d[e]), d[e] = fmaf(z.y, bf16_hi(__float_as_uint(w.z)), d[e]);
                d[e] = fmaf(z.z, bf16_lo(__float_as_uint(w.w)), d[e]), d[e] = fmaf(z.w, bf16_hi(__float_as_uint(w.w)), d[e]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int j = (i + (lane >> 1)) & 3;
                const float4 w = lds128f(f + (uint32_t)j * 16), x = up[j];
                d[e] = fmaf(x.x, w.x, d[e]), d[e] = fmaf(x.y, w.y, d[e]);
                d[e] = fmaf(x.z, w.z, d[e]), d[e] = fmaf(x.w, w.w, d[e]);
              }
            }
            d[e] *= __shfl_sync(0xffffffffu, row_sc, cc + e);
            // -0 changes no sum
            if (__shfl_sync(0xffffffffu, row_ad, cc + e) < 0) d[e] = -0.0f;
          }
          if (cc % C::RP == C::RP - 4) {
            // the slots have been read: the next rows' factors, or the next tile's
            named_bar_sync(1, kDecThreads);
            if (warp == 0 && !*abort_flag) {
              if (cc + 4 < C::CPW) ask(tile, cc / C::RP + 1);
              else if (q < n_it) ask(tile + 1, 0);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!ok || c0 + cc + e >= a.M || n >= NO) continue;
          const int64_t at = (int64_t)(c0 + cc + e) * NO + n;
          float w = v[e] + d[e];
          if (BWD && a.out_f32) {
            float* o = static_cast<float*>(a.y) + at;
            if (a.accumulate) w = *o + w;
            *o = w;
          } else {
            static_cast<uint16_t*>(a.y)[at] = f32_to_bf16_bits(w);
          }
        }
      }
      if (!head) {
        // every thread's stores, then the flag
        __threadfence();
        named_bar_sync(1, kDecThreads);
        if (threadIdx.x == 0) st_release_gpu(a.flags + u, 1u);
      }
    };

    // the first tile whose first step this CTA makes
    if (warp == 0 && (step0 == 0 ? n_it > 0 : n_it > S - step0)) ask(step0 == 0 ? tile0 : tile0 + 1, 0);
    // After a wait has given up, every warp still runs all its iterations,
    // without waiting: the epilogue's barriers count on all of them.
    auto iter = [&](Codes& f) {
      const int s = q & 1;
      if (q >= 2 && !*abort_flag && !mbar_wait(&empty[s], (uint32_t)((q >> 1) - 1) & 1u, DERR_TIMEOUT_BEMPTY))
        *abort_flag = 1u;
      if constexpr (!BWD) {
        tc_fence_after();  // of the products that read this stage
        __syncwarp();
      }
      decode(f, s);
      load(f);  // two steps ahead
      ++q;
    };
    for (int tile = tile0, step = step0; q < n_it; ++tile, step = 0) {
      const int len = min(S - step, n_it - q);
      // a segment that is followed by another is taken over once the first
      // step of that one is decoded: its products have long been made
      auto take = [&](int i) {
        if constexpr (BWD) {
          if (i > 0 && i % kGroup == 0 && group == kGroup) drain(i > kGroup);
        }
      };
      for (int i = 1; i < len; i += 2) {
        iter(f0);
        take(i - 1);
        iter(f1);
      }
      if (len & 1) {
        iter(f0);
        take(len - 1);
        const Codes f = f0;
        f0 = f1, f1 = f;
      }
      bool had = false;
      if constexpr (BWD) {
        had = len > group;
        if (had) drain(true);
      }
      epilogue(tile, step == 0, step + len == S, had);
    }
    if (!BWD && warp == 0 && *abort_flag) {  // copies in flight land first
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 200000ull) __nanosleep(1000);
    }
    if (!waited) {
      pdl_wait();
      pdl_launch_dependents();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kDecWarps) tmem_dealloc(tmem, C::TMEM_COLS);
}


// ------------------------------------------------------------------------ up to 16 rows, or a small weight
// The same product with mma.sync: a warp decodes 16 weight rows in registers,
// as the 16-row operand, and the rows of x are its 8-wide operand, so no decoded
// weight passes through shared memory and nothing is handed over.  A lane holds
// one 64-weight block of two weight rows per 256-deep step, so four lanes read
// a whole 128-byte line of codes; x is staged in shared memory in that order of
// k.  CTA = 128 weight rows; a cluster of CTAs shares their contraction and adds
// its partial sums in rank order through distributed shared memory.  Bound by
// the integer pipe too, with three CTAs an SM.
constexpr int kMmaWarps = 8;
constexpr int kMmaStages = 3;   // stages of x in flight
template <int NT>
struct MmaCfg {
  static constexpr int ROWS = kMmaWarps * 16;
  static constexpr int MR = NT * 8;
  static constexpr int SPS = NT <= 2 ? 2 : 1;      // 256-deep steps per stage of x
  static constexpr int STAGE = MR * 512 * SPS;     // bytes
  static constexpr int CTAS = NT <= 2 ? 3 : 2;  // CTAs of an SM that the registers allow
  static constexpr int PITCH = ROWS + 4;           // floats; [MR][PITCH] partial sums
  static constexpr int SMEM = kMmaStages * STAGE > MR * PITCH * 4 ? kMmaStages * STAGE : MR * PITCH * 4;
};

template <int NT, bool F16>
__global__ void __launch_bounds__(kMmaWarps * 32, MmaCfg<NT>::CTAS) k_few_mma(const FewArgs a) {
  using C = MmaCfg<NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = (int)lane_id(), warp = (int)warp_id(), g = lane >> 2, t = lane & 3;
  const int CS = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int m0 = (int)blockIdx.z * C::MR, mrows = min(C::MR, a.M - m0);
  const int n0 = (int)blockIdx.y * C::ROWS;
  // this warp's first weight row (a warp past the last row repeats the last
  // ones: its sums are not used)
  const int nw = min(n0 + warp * 16, a.N - 16);
  const int steps = (a.K + 255) / 256;
  const int s_beg = (int)((int64_t)rank * steps / CS), s_end = (int)((int64_t)(rank + 1) * steps / CS);

  // x of one stage: 16-byte chunk c (k = 8c ..) of row m of a 256-deep step at
  // chunk place (c % 8) * 4 + c / 8, odd rows with the 64-byte halves of each
  // 128 bytes swapped, so that the eight lanes of a quarter warp read eight
  // different bank groups.  A thread copies chunk xc of rows xm, xm + XM, ...
  constexpr int XC = 32 * C::SPS, XM = kMmaWarps * 32 / XC, XQ = C::MR / XM;
  static_assert(XQ >= 1 && C::MR % XM == 0, "every thread has a row");
  const int xc = threadIdx.x % XC, xm = threadIdx.x / XC;
  const uint16_t* xsrc = a.x + (int64_t)(m0 + xm) * a.K + (int64_t)s_beg * 256 + xc * 8;
  const uint32_t xdst = smem_u32(smem) + (uint32_t)((xc / 32) * C::MR * 512 + xm * 512 +
                                                    ((((xc & 7) * 4 + ((xc & 31) >> 3)) * 16) ^ ((xm & 1) * 64)));
  static_assert(XM % 2 == 0, "a thread's rows have one parity");
  int xk = s_beg * 256 + xc * 8;  // first element of the chunk
  const int xk_end = min(a.K, s_end * 256);
  auto stage_x = [&](int slot) {
    if (xk - xc * 8 < xk_end) {
#pragma unroll
      for (int q = 0; q < XQ; ++q) {
        const bool in = xm + q * XM < mrows && xk < xk_end;
        cp_async16(xdst + (uint32_t)(slot * C::STAGE + q * XM * 512), in ? xsrc + (int64_t)q * XM * a.K : a.x, in ? 16u : 0u);
      }
      xsrc += 256 * C::SPS;
      xk += 256 * C::SPS;
    }
    cp_async_commit();
  };
  // codes and scales of the step to come, reloaded as they are used
  uint4 cw[2][2];
  float cs[2];
  const int64_t kb = a.K / 2;
  const uint8_t* cp = a.codes + (int64_t)(nw + g) * kb + (int64_t)s_beg * 128 + t * 32;
  const float* sp = a.absmax + ((int64_t)s_beg * 4 + t) * a.N + nw + g;
  // the last step may end inside its four blocks: lanes past the end read
  // codes that exist and a scale of 0
  int k_lane = s_beg * 256 + t * 64;
  auto load_w = [&](int q) {
    const uint8_t* p = k_lane < a.K ? cp : a.codes;
#pragma unroll
    for (int h = 0; h < 2; ++h) cw[h][q] = __ldg(reinterpret_cast<const uint4*>(p + (int64_t)(h * 8) * kb) + q);
  };
  auto load_s = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h) cs[h] = k_lane < a.K ? __ldg(sp + h * 8) : 0.0f;
  };
#pragma unroll
  for (int i = 0; i < kMmaStages - 1; ++i) stage_x(i);
  if (s_beg < s_end) {
    load_s();
    load_w(0);
    load_w(1);
  }
  float acc[NT][4] = {};
  int slot = 0, part = 0;  // stage of x and step within it
  for (int s = s_beg; s < s_end; ++s) {
    if (part == 0) {
      cp_async_wait<kMmaStages - 2>();
      __syncthreads();  // this stage of x has landed; everyone is done with the one before
      stage_x(slot == 0 ? kMmaStages - 1 : slot - 1);
    }
    Nf4Table tb[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) tb[h] = make_table(cs[h]);
    const bool more = s + 1 < s_end;
    const int k_now = k_lane;
    cp += 128;
    sp += (int64_t)4 * a.N;
    k_lane = k_now + 256;
    if (more) load_s();
    const uint8_t* xs = smem + slot * C::STAGE + part * C::MR * 512 + g * 512 + t * 16;
    const uint32_t flip = (uint32_t)(g & 1) * 64;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      uint4 d[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 q = cw[h][w / 4];
        const uint32_t c = (w & 3) == 0 ? q.x : (w & 3) == 1 ? q.y : (w & 3) == 2 ? q.z : q.w;
        d[h] = dq8(c, tb[h]);
      }
      if ((w & 3) == 3 && more) load_w(w / 4);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 b = *reinterpret_cast<const uint4*>(xs + nt * 4096 + ((w * 64) ^ flip));
        mma16816(acc[nt], d[0].x, d[1].x, d[0].y, d[1].y, b.x, b.y);
        mma16816(acc[nt], d[0].z, d[1].z, d[0].w, d[1].w, b.z, b.w);
      }
    }
    if (++part == C::SPS) {
      part = 0;
      if (++slot == kMmaStages) slot = 0;
    }
  }
  cp_async_wait<0>();
  __syncthreads();
  // partial sums [m][n]
  float* red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      red[(nt * 8 + 2 * t + (e & 1)) * C::PITCH + warp * 16 + (e >> 1) * 8 + g] = acc[nt][e];
  // U, and y's earlier readers, are an earlier kernel's business until here
  pdl_wait();
  pdl_launch_dependents();
  if (CS > 1) cluster_sync();
  else __syncthreads();
  // the cluster's threads share the results out, two columns each at a time
  for (int i = rank * kMmaWarps * 32 + (int)threadIdx.x; i < C::ROWS / 2 * mrows; i += CS * kMmaWarps * 32) {
    const int m = i / (C::ROWS / 2), nl = 2 * (i % (C::ROWS / 2)), n = n0 + nl;
    if (n >= a.N) continue;
    float v0 = 0.0f, v1 = 0.0f;
    for (int c = 0; c < CS; ++c) {
      float p0, p1;
      asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                   : "=f"(p0), "=f"(p1)
                   : "r"(mapa_shared(smem_u32(&red[m * C::PITCH + nl]), (uint32_t)c))
                   : "memory");
      v0 += p0;
      v1 += p1;
    }
    const int ad = a.row[m0 + m];
    if (ad >= 0) {
      const float s = a.scale[ad];
      const float4* u = reinterpret_cast<const float4*>(a.P + (int64_t)(m0 + m) * 16);
      float d0 = 0.0f, d1 = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 uu = u[q];
        float b0[4], b1[4];
        const int64_t o = ad * a.stride + (int64_t)n * 16 + 4 * q;
        if constexpr (F16) {
          const uint2 x0 = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.F) + o));
          const uint2 x1 = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.F) + o + 16));
          b0[0] = bf16_lo(x0.x), b0[1] = bf16_hi(x0.x), b0[2] = bf16_lo(x0.y), b0[3] = bf16_hi(x0.y);
          b1[0] = bf16_lo(x1.x), b1[1] = bf16_hi(x1.x), b1[2] = bf16_lo(x1.y), b1[3] = bf16_hi(x1.y);
        } else {
          const float4 x0 = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.F) + o));
          const float4 x1 = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.F) + o + 16));
          b0[0] = x0.x, b0[1] = x0.y, b0[2] = x0.z, b0[3] = x0.w;
          b1[0] = x1.x, b1[1] = x1.y, b1[2] = x1.z, b1[3] = x1.w;
        }
        d0 = fmaf(uu.x, b0[0], d0), d0 = fmaf(uu.y, b0[1], d0), d0 = fmaf(uu.z, b0[2], d0), d0 = fmaf(uu.w, b0[3], d0);
        d1 = fmaf(uu.x, b1[0], d1), d1 = fmaf(uu.y, b1[1], d1), d1 = fmaf(uu.z, b1[2], d1), d1 = fmaf(uu.w, b1[3], d1);
      }
      v0 = fmaf(s, d0, v0);
      v1 = fmaf(s, d1, v1);
    }
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.y) + (int64_t)(m0 + m) * a.N + n) = pack_bf16x2(v0, v1);
  }
  if (CS > 1) cluster_sync();  // the sums stay until every CTA of the cluster has read them
}

template <int NT, bool F16>
cudaError_t launch_mma(const FewArgs& a, cudaStream_t st) {
  using C = MmaCfg<NT>;
  auto k = k_few_mma<NT, F16>;
  static const cudaError_t attr = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (attr != cudaSuccess) return attr;
  const int blocks = (a.N + C::ROWS - 1) / C::ROWS, chunks = (a.M + C::MR - 1) / C::MR, steps = (a.K + 255) / 256;
  // CTAs sharing a contraction: the shortest time of the busiest SM, in tenths
  // of a step's decoding.  One or two CTAs leave part of the SM idle (k steps
  // side by side take 2.2, 2.8 and 3, 4, ... steps' time), and a CTA counts
  // about a step to start and join.
  int cs = 1;
  int64_t best = INT64_MAX;
  for (int c = 1; c <= 8; ++c) {
    const int64_t per_sm = ((int64_t)blocks * chunks * c + device_sm_count() - 1) / device_sm_count();
    const int64_t cost = (per_sm == 1 ? 22 : per_sm == 2 ? 28 : 10 * per_sm) * ((steps + c - 1) / c + 1);
    if (cost <= best) best = cost, cs = c;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cs, (unsigned)blocks, (unsigned)chunks);
  cfg.blockDim = dim3(kMmaWarps * 32);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = (unsigned)cs;
  attrs[0].val.clusterDim.y = 1;
  attrs[0].val.clusterDim.z = 1;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, k, a);
}

template <int NX, bool BWD, bool F16>
cudaError_t launch(FewArgs a, cudaStream_t st) {
  using C = Cfg<NX, BWD, F16>;
  static const cudaError_t attr =
      cudaFuncSetAttribute(k_few<NX, BWD, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (attr != cudaSuccess) return attr;
  const int kc = BWD ? a.N : a.K, no = BWD ? a.K : a.N;  // contraction, outputs
  const int blocks = (no + kRows - 1) / kRows;
  a.steps = (kc + 255) / 256;
  CUtensorMap tm;
  if (!tmap_bf16_sw128(&tm, a.x, (uint64_t)kc, (uint64_t)a.M, (uint64_t)kc * 2, 64, NX)) return cudaErrorInvalidValue;
  const int64_t iters = (int64_t)blocks * a.steps;
  int64_t grid = device_sm_count() < kFewUnits ? device_sm_count() : kFewUnits;
  if (grid > iters) grid = iters;
  if (iters >= (1ll << 31)) return cudaErrorInvalidValue;
  a.base = (int)(iters / grid);
  a.extra = (int)(iters % grid);
  note_launch();
  return launch_pdl(k_few<NX, BWD, F16>, dim3((unsigned)grid), dim3(kFewThreads), C::SMEM, st, tm, a);
}

}  // namespace

namespace {
template <bool F16>
cudaError_t run_few_t(const FewArgs& a, cudaStream_t st) {
  const bool fits = a.N <= 65535 * kMmaWarps * 16;  // k_few_mma's grid holds that many tiles
  if (a.M <= 8 && fits) return launch_mma<1, F16>(a, st);
  if (a.M <= 16 && fits) return launch_mma<2, F16>(a, st);
  // With more rows mma.sync's own rate and its reads of x bind: k_few is ahead
  // once it has several steps for every SM to make good its joins (32 rows,
  // k_few / k_few_mma: 3584x3584 16 / 13 us, 5120x5120 20 / 24 us, 27648x5120
  // 52 / 62 us; 64 rows: 22 / 20, 25 / 37, 62 / 103 us).
  const int64_t steps = (int64_t)((a.N + 127) / 128) * ((a.K + 255) / 256);
  if (steps >= 4 * device_sm_count())
    return a.M <= 32 ? launch<32, false, F16>(a, st) : launch<64, false, F16>(a, st);
  return a.M <= 32 ? launch_mma<4, F16>(a, st) : launch_mma<8, F16>(a, st);
}
}  // namespace

cudaError_t run_few(const FewArgs& a, bool f16, cudaStream_t st) {
  return f16 ? run_few_t<true>(a, st) : run_few_t<false>(a, st);
}

cudaError_t run_few_bwd(const FewArgs& a, cudaStream_t st) {
  return a.M <= 32 ? launch<32, true, false>(a, st) : launch<64, true, false>(a, st);
}

}  // namespace ws
