// lora_few.cu -- forward of the many-adapter NF4 linear for few rows (decode):
// y = x W'^T + the adapter term, up to 64 rows at a time.
//
// Bound by decoding the codes (about three integer instructions a weight, on a
// pipe of 64 lanes an SM), then by reading them.  The dequant GEMM's tile has
// the activation rows as the 128-row operand and hands over 64-deep steps; with
// few rows its time is that handshake.  Here the WEIGHT rows are the 128-row
// operand and the rows of x the N-wide one (16, 32 or 64), and a step is 256
// deep: sixteen warps decode 128 x 256 weights, each thread one 64-weight block
// (one value table for 64 weights), straight into the 128-byte swizzled operand
// layout, then hand over once; one thread loads x by TMA and issues the
// tensor-core products (tcgen05, fp32 sums in tensor memory) of one step while
// the next is decoded.
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

template <int NX>
struct Cfg {
  static constexpr uint32_t X_BYTES = NX * 512;  // a step of x: four sub-tiles of NX rows
  static constexpr int XS = NX == 64 ? 3 : 4;    // steps of x in flight
  static constexpr uint32_t OFF_A = 0, OFF_X = 2 * kABytes, OFF_BAR = OFF_X + XS * X_BYTES;
  static constexpr uint32_t SMEM = OFF_BAR + 192 + 1024;  // + alignment slack
  static_assert(SMEM <= 227u * 1024u, "shared memory");
  static constexpr uint32_t TMEM_COLS = NX < 32 ? 32 : NX;
  static constexpr int CPW = NX / 4;             // accumulator columns (rows of x) of one epilogue warp
};

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

template <int NX, bool F16>
__global__ void __launch_bounds__(kFewThreads, 1)
    k_few(const __grid_constant__ CUtensorMap tmX, const FewArgs a) {
  using C = Cfg<NX>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [2] a step's weights are there
  uint64_t* empty = full + 2;                                       // [2] ... and have been used
  uint64_t* xfull = empty + 2;                                      // [XS] the same for x
  uint64_t* xempty = xfull + C::XS;
  uint64_t* acc_done = xempty + C::XS;                              // a piece's sums are complete
  uint64_t* acc_free = acc_done + 1;                                // ... and have been read
  uint32_t* misc = reinterpret_cast<uint32_t*>(acc_free + 1);
  volatile uint32_t* abort_flag = misc + 1;
  volatile uint32_t* got_flag = misc + 2;
  // (the shuffle tells the compiler that a warp's index is one value)
  const int warp = __shfl_sync(0xffffffffu, (int)warp_id(), 0), lane = (int)lane_id();
  const int T = a.blocks * a.chunks, S = a.steps;
  const int64_t I = (int64_t)T * S, U = gridDim.x, u = blockIdx.x;
  const int64_t pb = u * I / U, pe = (u + 1) * I / U;
  if (threadIdx.x == 0) {
    *abort_flag = *(volatile uint32_t*)&g_dev_error;  // an earlier kernel gave up: do nothing
    for (int s = 0; s < 2; ++s) {
      mbar_init(&full[s], kDecWarps);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < C::XS; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], 1);
    }
    mbar_init(acc_done, 1);
    mbar_init(acc_free, kDecWarps);
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
  const int n_it = skip ? 0 : (int)(pe - pb);

  if (warp == kDecWarps) {
    // ------------------------------------------------------------ the products
    // The whole warp runs the loop and one lane issues: descriptors then stay
    // in uniform registers (issued from a single-lane branch, a step's sixteen
    // products took 2000 cycles to issue, as long as decoding it).
    const bool leader = elect_one();
    constexpr uint32_t idesc = idesc_bf16_f32(kRows, NX, 0u);
    const uint64_t ad0 = smem_desc_sw128(smem_u32(smem + C::OFF_A), 16, 1024);
    const uint64_t bd0 = smem_desc_sw128(smem_u32(smem + C::OFF_X), 16, 1024);
    int step = (int)(pb % S), xs = 0;
    uint32_t pieces = 0, xph = 0;
    bool first = true;  // of its piece
    for (int q = 0; q < n_it; ++q) {
      const int s = q & 1;
      bool ok = *abort_flag == 0u && mbar_wait(&full[s], (uint32_t)(q >> 1) & 1u, DERR_TIMEOUT_FULL) &&
                mbar_wait(&xfull[xs], xph, DERR_TIMEOUT_FULL) &&
                !(first && pieces > 0 && !mbar_wait(acc_free, (pieces - 1) & 1u, DERR_TIMEOUT_ACC));
      if (!__all_sync(0xffffffffu, ok)) {
        *abort_flag = 1u;
        break;
      }
      tc_fence_after();
      const bool end = ++step == S || q + 1 == n_it;
      if (leader) {
        const uint64_t ad = ad0 + (uint64_t)(s * (kABytes >> 4));
        const uint64_t bd = bd0 + (uint64_t)(xs * (C::X_BYTES >> 4));
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_f16(tmem, ad + (uint64_t)(t * 1024 + 2 * k), bd + (uint64_t)(t * NX * 8 + 2 * k), idesc,
                       (t > 0 || k > 0 || !first) ? 1u : 0u);
        tc_commit(&empty[s]);
        tc_commit(&xempty[xs]);
        if (end) tc_commit(acc_done);
      }
      __syncwarp();
      if (++xs == C::XS) {
        xs = 0;
        xph ^= 1u;
      }
      first = end;
      if (end) {
        step = 0;
        ++pieces;
      }
    }
    // every product has completed before tensor memory is freed (the last
    // piece's commit covers all before it)
    if (pieces > 0) mbar_wait(acc_done, (pieces - 1) & 1u, DERR_TIMEOUT_DRAIN);
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
      int tile = (int)(pb / S), step = (int)(pb % S), xs = 0;
      uint32_t ph = 1;
      for (int q = 0; q < n_it; ++q) {
        if (*abort_flag || !mbar_wait(&xempty[xs], ph, DERR_TIMEOUT_EMPTY)) {
          *abort_flag = 1u;
          break;
        }
        mbar_arrive_expect_tx(&xfull[xs], C::X_BYTES);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          tma_load_2d(smem + C::OFF_X + xs * C::X_BYTES + t * (NX * 128), &tmX, &xfull[xs], step * 256 + t * 64,
                      tile / a.blocks * NX);
        if (++xs == C::XS) {
          xs = 0;
          ph ^= 1u;
        }
        if (++step == S) {
          step = 0;
          ++tile;
        }
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
    // Thread = weight row r of the tile, 64-weight block t of the step (four
    // lanes read a 128-byte line of codes).  It takes its eight 8-weight words
    // from word 2t on, so that the eight lanes of a quarter warp (two rows,
    // four blocks) store to eight different 16-byte places of the swizzle.
    const int r = (int)threadIdx.x >> 2, t = (int)threadIdx.x & 3;
    uint32_t dst[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      dst[i] = smem_u32(smem + C::OFF_A) + (uint32_t)(t * 16384 + r * 128 + ((((i + 2 * t) & 7) ^ (r & 7)) << 4));
    struct Codes {
      uint2 w[4];
      float s;
    };
    const int64_t kb = a.K / 2;
    int lt = (int)(pb / S), ls = (int)(pb % S), left = n_it;  // next step to load
    const uint8_t* cp = nullptr;
    const float* sp = nullptr;
    auto seek = [&]() {
      // rows past the last repeat it: their sums are not stored
      const int n = min(lt % a.blocks * kRows + r, a.N - 1);
      cp = a.codes + n * kb + (int64_t)ls * 128 + t * 32;
      sp = a.absmax + ((int64_t)ls * 4 + t) * a.N + n;
    };
    auto load = [&](Codes& f) {
      if (left <= 0) return;
      // the last step may end inside its four blocks: blocks past the end take
      // codes that exist and a scale of 0
      const bool in = ls * 256 + t * 64 < a.K;
      const uint2* c = reinterpret_cast<const uint2*>(in ? cp : a.codes);
#pragma unroll
      for (int i = 0; i < 4; ++i) f.w[i] = __ldg(c + ((i + t) & 3));
      f.s = in ? __ldg(sp) : 0.0f;
      --left;
      if (++ls == S) {
        ls = 0;
        ++lt;
        seek();
      } else {
        cp += 128;
        sp += (int64_t)4 * a.N;
      }
    };
    auto decode = [&](const Codes& f, int s) {
      const Nf4Table tb = make_table(f.s);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 v = dq8((i & 1) ? f.w[i / 2].y : f.w[i / 2].x, tb);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst[i] + (uint32_t)s * kABytes), "r"(v.x),
                     "r"(v.y), "r"(v.z), "r"(v.w)
                     : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
    };
    bool waited = false;  // for the earlier kernels
    uint32_t piece = 0;
    // The piece that ends with iteration q: tile `tile`, whether it holds the
    // tile's first and its last step.
    auto epilogue = [&](int tile, bool head, bool tail) {
      const bool ok = !*abort_flag && mbar_wait_backoff(acc_done, piece & 1u, DERR_TIMEOUT_ACC);
      ++piece;
      if (!ok) *abort_flag = 1u;
      tc_fence_after();
      if (!waited) {
        pdl_wait();
        pdl_launch_dependents();
        waited = true;
      }
      const int q4 = warp & 3, c0 = warp / 4 * C::CPW;  // lanes (weight rows) and columns of this warp
      const int nl = q4 * 32 + lane, n = tile % a.blocks * kRows + nl;
      const int m0 = tile / a.blocks * NX + c0;
      int64_t last = u;  // CTA that holds the tile's last step
      if (head && !tail) {
        last = ((int64_t)(tile + 1) * S * U - 1) / I;
        if (threadIdx.x == 0) {
          bool got = ok;
          for (int64_t v = u + 1; v <= last && got; ++v) {
            got = wait_flag_bounded(a.flags + v, 1u, kWaitLimitNs, DERR_TIMEOUT_PEER);
          }
          *got_flag = got ? 1u : 0u;
        }
        named_bar_sync(1, kDecThreads);
        if (*got_flag == 0u) last = u;
      }
#pragma unroll
      for (int cc = 0; cc < C::CPW; cc += 4) {
        uint32_t raw[4];
        tmem_ld_x4(tmem + ((uint32_t)(q4 * 32) << 16) + (uint32_t)(c0 + cc), raw);
        tmem_ld_wait();
        if (cc + 4 == C::CPW) {  // the sums are in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_free);
        }
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(raw[e]);
        if (!head) {  // a later piece of its tile: hand it over
          float* p = a.partial + (u * NX + c0 + cc) * kRows + nl;
#pragma unroll
          for (int e = 0; e < 4; ++e) __stcg(p + e * kRows, v[e]);
          continue;
        }
        // later pieces in step order, four at a time in flight
        for (int64_t w = u + 1; w <= last; w += 4) {
          float x[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float* p = a.partial + ((w + i) * NX + c0 + cc) * kRows + nl;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] = w + i <= last ? __ldcg(p + e * kRows) : 0.0f;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += x[i][e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int m = m0 + cc + e;
          if (!ok || m >= a.M || n >= a.N) continue;
          const int ad = a.row[m];
          if (ad >= 0) {
            const float4* up = reinterpret_cast<const float4*>(a.P + (int64_t)m * 16);
            float d = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 uu = up[j];
              float b[4];
              const int64_t o = ad * a.stride + (int64_t)n * 16 + 4 * j;
              if constexpr (F16) {
                const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.F) + o);
                b[0] = bf16_lo(x.x), b[1] = bf16_hi(x.x), b[2] = bf16_lo(x.y), b[3] = bf16_hi(x.y);
              } else {
                const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.F) + o);
                b[0] = x.x, b[1] = x.y, b[2] = x.z, b[3] = x.w;
              }
              d = fmaf(uu.x, b[0], d), d = fmaf(uu.y, b[1], d), d = fmaf(uu.z, b[2], d), d = fmaf(uu.w, b[3], d);
            }
            v[e] = fmaf(a.scale[ad], d, v[e]);
          }
          a.y[(int64_t)m * a.N + n] = f32_to_bf16_bits(v[e]);
        }
      }
      if (!head) {
        // every thread's stores, then the flag
        __threadfence();
        named_bar_sync(1, kDecThreads);
        if (threadIdx.x == 0) st_release_gpu(a.flags + u, 1u);
      }
    };

    int tile = lt, step = ls;
    bool head = ls == 0;  // of the piece being made
    Codes f0{}, f1{};
    seek();
    load(f0);
    load(f1);
    // After a wait has given up, every warp still runs all its iterations,
    // without waiting: the epilogue's barriers count on all of them.
    auto iter = [&](int q, Codes& f, int s) {
      if (q >= 2 && !*abort_flag && !mbar_wait(&empty[s], (uint32_t)((q >> 1) - 1) & 1u, DERR_TIMEOUT_BEMPTY))
        *abort_flag = 1u;
      decode(f, s);
      load(f);  // two steps ahead
      const bool tail = ++step == S;
      if (tail || q + 1 == n_it) {
        epilogue(tile, head, tail);
        head = true;
        step = 0;
        ++tile;
      }
    };
    for (int q = 0; q < n_it; q += 2) {
      iter(q, f0, 0);
      if (q + 1 < n_it) iter(q + 1, f1, 1);
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

template <int NX, bool F16>
cudaError_t launch(FewArgs a, cudaStream_t st) {
  using C = Cfg<NX>;
  static const cudaError_t attr =
      cudaFuncSetAttribute(k_few<NX, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (attr != cudaSuccess) return attr;
  a.blocks = (a.N + kRows - 1) / kRows;
  a.chunks = (a.M + NX - 1) / NX;
  a.steps = (a.K + 255) / 256;
  CUtensorMap tm;
  if (!tmap_bf16_sw128(&tm, a.x, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)a.K * 2, 64, NX)) return cudaErrorInvalidValue;
  const int64_t iters = (int64_t)a.blocks * a.chunks * a.steps;
  int64_t grid = device_sm_count() < kFewUnits ? device_sm_count() : kFewUnits;
  if (grid > iters) grid = iters;
  note_launch();
  return launch_pdl(k_few<NX, F16>, dim3((unsigned)grid), dim3(kFewThreads), C::SMEM, st, tm, a);
}

}  // namespace

cudaError_t run_few(const FewArgs& a, bool f16, cudaStream_t st) {
  if (a.M <= 16) return f16 ? launch<16, true>(a, st) : launch<16, false>(a, st);
  if (a.M <= 32) return f16 ? launch<32, true>(a, st) : launch<32, false>(a, st);
  return f16 ? launch<64, true>(a, st) : launch<64, false>(a, st);
}

}  // namespace ws
