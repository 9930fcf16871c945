// adamw.cu -- one AdamW step over many tensors (decoupled weight decay,
// Loshchilov & Hutter, 2019), moments in 32 bits or in 8, with the global
// gradient norm of each parameter group and clipping by it.
//
// All tensors of a plan run in one launch: the plan cuts every tensor into
// chunks of kChunk elements and lists the chunks by group; CTA c works on
// chunk c.  Every operand is read once
// and written once; each element needs the group's coefficients only, so the
// step is bound by memory (28 bytes per fp32 parameter with 32-bit states,
// 16 with 8-bit ones).
//
// Sums of squares run in a fixed order in two fp32 parts (16 elements of a
// thread, a butterfly, 8 warps; then the chunks the same way), so repeated steps
// give the same bits and the clip factor is the rounded one of exact sums.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <vector>

#include "common.cuh"
#include "kernels.h"

namespace ws {

namespace {

constexpr int kChunk = 4096;   // elements per CTA: 16 per thread, all loads in flight at once
constexpr int kThreads = 256;
constexpr int kBlock8 = 256;   // elements per 8-bit state block: one warp, 8 per lane

// One chunk of the plan's device image (64 bytes): the addresses of its first
// elements, so that a CTA's data is one load away.
struct Chunk {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int32_t n;  // elements, 1 .. kChunk
  int32_t group;
  int32_t pad[2];
};
static_assert(sizeof(Chunk) == 64, "chunk entry");

// Coefficients of a group's step, written by k_adamw_begin.
struct Coef {
  float beta1, one_m_beta1, beta2, one_m_beta2;
  float decay;      // 1 - lr * weight_decay
  float step_size;  // lr / (1 - beta1^t)
  float rbc2;       // 1 / sqrt(1 - beta2^t)
  float eps;
  float clip;       // gradient factor
  int32_t skip;     // the group takes no step
  int32_t pad[2];
};
static_assert(sizeof(Coef) == 48, "coefficients");

size_t al16(size_t x) { return (x + 15) & ~size_t(15); }

// Sections of the plan image: the chunks listed by group, and the first chunk
// of each group (n_groups + 1 entries).
struct Layout {
  size_t chunk, group_first, bytes;
};
Layout plan_layout(int32_t n_groups, int64_t n_chunks) {
  Layout L{};
  L.chunk = 0;
  L.group_first = (size_t)n_chunks * sizeof(Chunk);
  L.bytes = L.group_first + al16((size_t)(n_groups + 1) * 4);
  return L;
}
size_t coef_bytes(int32_t n_groups) { return al16((size_t)n_groups * sizeof(Coef)); }

// ---- 8-bit codes ------------------------------------------------------------------
// First moment: e4m3, two values per conversion, saturating at 448.
WS_DEVINL uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
WS_DEVINL void e4m3x2_to_f32(uint32_t v, float& lo, float& hi) {
  uint32_t h;  // two f16
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}
// Root of the second moment: unsigned, 4 exponent and 4 mantissa bits,
// (1 + (c & 15) / 16) 2^((c >> 4) - 15); code 0 is 0 and a non-zero root gets
// at least code 1, so a denominator never collapses to eps because its
// element is small beside its block's largest.  The code is the fp32 pattern
// rounded to 4 mantissa bits (ties to even) with its exponent rebased: one
// bit more than e4m3 has, for the sign a root does not need.
constexpr uint32_t kRootBias = (127u - 15u) << 4;
WS_DEVINL uint32_t root_code(float q) {
  const uint32_t b = __float_as_uint(q);  // q >= 0
  const int r = (int)(b + ((b >> 19) & 1u) + (0x3FFFFu - (kRootBias << 19))) >> 19;
  return (uint32_t)max(r, (int)min(b, 1u));  // (NaN: nonsense, in a block whose scale is not finite)
}
WS_DEVINL float root_value(uint32_t c) {
  return c ? __uint_as_float(c * (1u << 19) + (kRootBias << 19)) : 0.0f;
}
constexpr float kMTop = 448.0f, kVTop = 1.9375f;

// ---- elements ------------------------------------------------------------------------
// N (4 or 8) consecutive elements from i0 of an fp32 or bf16 array of n; past
// the end they read as 0 and are not written.  Full vectors use 32-byte
// (fp32 x 8, where aligned), 16-byte or (bf16 x 4) 8-byte accesses.
template <bool BF16, int N>
WS_DEVINL void load_n(const void* base, int i0, int n, float (&x)[N]) {
  if (i0 + N <= n) {
    if constexpr (BF16) {
      const uint32_t* s = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(base) + i0);
      uint32_t w[N / 2];
      if constexpr (N == 8) {
        const uint4 q = *reinterpret_cast<const uint4*>(s);
        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
      } else {
        const uint2 q = *reinterpret_cast<const uint2*>(s);
        w[0] = q.x, w[1] = q.y;
      }
#pragma unroll
      for (int k = 0; k < N / 2; ++k) x[2 * k] = bf16_lo(w[k]), x[2 * k + 1] = bf16_hi(w[k]);
    } else {
      const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i0);
      if constexpr (N == 8) {
        // one 32-byte access: two of 16 bytes would each touch half of every sector
        if ((reinterpret_cast<uintptr_t>(s) & 31u) == 0u) {
          uint32_t w[8];
          ld_global_v8(s, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(w[k]);
          return;
        }
      }
#pragma unroll
      for (int k = 0; k < N / 4; ++k) {
        const float4 q = s[k];
        x[4 * k] = q.x, x[4 * k + 1] = q.y, x[4 * k + 2] = q.z, x[4 * k + 3] = q.w;
      }
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    x[k] = 0.0f;
    if (i0 + k < n)
      x[k] = BF16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(base)[i0 + k])
                  : static_cast<const float*>(base)[i0 + k];
  }
}
template <bool BF16, int N>
WS_DEVINL void store_n(void* base, int i0, int n, const float (&x)[N]) {
  if (i0 + N <= n) {
    if constexpr (BF16) {
      uint32_t w[N / 2];
#pragma unroll
      for (int k = 0; k < N / 2; ++k) w[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
      uint16_t* d = static_cast<uint16_t*>(base) + i0;
      if constexpr (N == 8) *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
      else *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
    } else {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + i0);
      if constexpr (N == 8) {
        if ((reinterpret_cast<uintptr_t>(d) & 31u) == 0u) {
          st_global_v8(d, __float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]),
                       __float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
          return;
        }
      }
#pragma unroll
      for (int k = 0; k < N / 4; ++k) d[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (i0 + k < n) {
      if constexpr (BF16) static_cast<uint16_t*>(base)[i0 + k] = f32_to_bf16_bits(x[k]);
      else static_cast<float*>(base)[i0 + k] = x[k];
    }
}

WS_DEVINL float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

WS_DEVINL float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// m, v and p of one element.  Products and sums are rounded one by one (no
// contraction), as the formula is written: a value that lies on the border
// between two 8-bit codes then falls the way it does for anybody who
// evaluates the formula in fp32.
// Returns the root of the new v, correctly rounded (EXACT: it is kept, as an
// 8-bit code) or to 2^-22.
template <bool EXACT>
WS_DEVINL float adamw1(float& p, float g, float& m, float& v, const Coef& c) {
  g = __fmul_rn(g, c.clip);
  m = __fadd_rn(__fmul_rn(m, c.beta1), __fmul_rn(g, c.one_m_beta1));
  v = __fadd_rn(__fmul_rn(v, c.beta2), __fmul_rn(__fmul_rn(g, g), c.one_m_beta2));
  // the step to 2^-21 or better: it is a small change of p
  const float root = EXACT ? __fsqrt_rn(v) : sqrt_approx(v);
  p = fmaf(-c.step_size, m * rcp_approx(fmaf(root, c.rbc2, c.eps)), p * c.decay);
  return root;
}

// ---- kernels ---------------------------------------------------------------------------
// Only the plan's tables are declared __restrict__: what an earlier kernel
// writes may not be, or the compiler may load it ahead of the wait for that
// kernel.
// A sum in two fp32 parts, h + l: twice the precision at a few operations an
// addition, where double precision would bind the pass (Knuth's two-sum, and a
// product's error by a fused multiply-add).
struct Sum2 {
  float h, l;
};
WS_DEVINL void add2(Sum2& s, float x) {
  const float t = __fadd_rn(s.h, x), z = __fsub_rn(t, s.h);
  s.l = __fadd_rn(s.l, __fadd_rn(__fsub_rn(s.h, __fsub_rn(t, z)), __fsub_rn(x, z)));
  s.h = t;
}
WS_DEVINL void add2(Sum2& s, float x, float e) {
  add2(s, x);
  s.l = __fadd_rn(s.l, e);
}
WS_DEVINL Sum2 warp_sum2(Sum2 s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float h = __shfl_xor_sync(0xffffffffu, s.h, o), l = __shfl_xor_sync(0xffffffffu, s.l, o);
    add2(s, h, l);  // (a NaN stays)
  }
  return s;
}

// A CTA takes kSumChunks chunks, all their loads in flight at once.
constexpr int kSumChunks = 4;
template <bool G16>
__global__ void __launch_bounds__(kThreads)
    k_adamw_sumsq(const Chunk* __restrict__ chunks, int n_chunks, float2* partial) {
  __shared__ Sum2 red[kSumChunks][kThreads / 32];
  const int c0 = (int)blockIdx.x * kSumChunks;
  const void* gp[kSumChunks];
  int n[kSumChunks];
#pragma unroll
  for (int c = 0; c < kSumChunks; ++c) {
    const bool in = c0 + c < n_chunks;
    gp[c] = in ? chunks[c0 + c].g : nullptr;
    n[c] = in ? chunks[c0 + c].n : 0;
  }
  pdl_wait();
  pdl_launch_dependents();
  float g[kSumChunks][2][8];
#pragma unroll
  for (int c = 0; c < kSumChunks; ++c)
#pragma unroll
    for (int u = 0; u < 2; ++u) load_n<G16, 8>(gp[c], (u * kThreads + (int)threadIdx.x) * 8, n[c], g[c][u]);
#pragma unroll
  for (int c = 0; c < kSumChunks; ++c) {
    Sum2 s{0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float x = g[c][u][k], q = __fmul_rn(x, x);
        if (G16) add2(s, q);  // (the square of a bf16 value is exact)
        else add2(s, q, fmaf(x, x, -q));
      }
    s = warp_sum2(s);
    if (lane_id() == 0) red[c][warp_id()] = s;
  }
  __syncthreads();
  if (threadIdx.x < kSumChunks && c0 + (int)threadIdx.x < n_chunks) {
    Sum2 s = red[threadIdx.x][0];
    for (int w = 1; w < kThreads / 32; ++w) add2(s, red[threadIdx.x][w].h, red[threadIdx.x][w].l);
    partial[c0 + threadIdx.x] = make_float2(s.h, s.l);
  }
}

// b^t for an integer t, by squaring.
WS_DEVINL double pow_int(double b, double t) {
  uint32_t n = (uint32_t)fmin(t, 4e9);
  double r = 1.0;
  for (; n; n >>= 1, b *= b)
    if (n & 1u) r *= b;
  return r;
}

// One CTA per group: the norm from the chunks' sums, the step counter and the
// coefficients.  A thread adds its chunks (every kBeginThreads-th) in order, a
// butterfly and then the warps in index order follow.  Double precision is
// slow here (a warp's product takes as long as dozens in fp32: with every
// thread computing the powers the kernel took 25 us), so only one thread each
// makes them and the sums stay in fp32 parts.
constexpr int kBeginThreads = 1024;
__global__ void __launch_bounds__(kBeginThreads)
    k_adamw_begin(ws_adamw_group* groups, const int32_t* __restrict__ group_first,
                  const float2* partial, float* norms, int clip,
                  Coef* coef) {
  __shared__ Sum2 red[kBeginThreads / 32];
  __shared__ float bc[2];  // 1 - beta^t
  const int h = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  if (partial) {
    Sum2 s{0.0f, 0.0f};
    const int end = group_first[h + 1];
    int i = group_first[h] + threadIdx.x;
    for (; i + 3 * kBeginThreads < end; i += 4 * kBeginThreads) {
      const float2 a = partial[i], b = partial[i + kBeginThreads], c = partial[i + 2 * kBeginThreads],
                   d = partial[i + 3 * kBeginThreads];
      add2(s, a.x, a.y);
      add2(s, b.x, b.y);
      add2(s, c.x, c.y);
      add2(s, d.x, d.y);
    }
    for (; i < end; i += kBeginThreads) add2(s, partial[i].x, partial[i].y);
    s = warp_sum2(s);
    if (lane_id() == 0) red[warp_id()] = s;
  }
  if (threadIdx.x == 32 || threadIdx.x == 64) {
    const double b = threadIdx.x == 32 ? groups[h].beta1 : groups[h].beta2;
    bc[threadIdx.x / 32 - 1] = (float)(1.0 - pow_int(b, groups[h].step + 1.0));
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  const ws_adamw_group g = groups[h];
  Coef c{};
  c.clip = 1.0f;
  if (partial) {
    Sum2 s = red[0];
    for (int w = 1; w < kBeginThreads / 32; ++w) add2(s, red[w].h, red[w].l);
    // (a sum that is not finite has no error part)
    const double norm = isfinite(s.h) ? sqrt((double)s.h + (double)s.l) : (double)s.h;
    if (norms) norms[h] = (float)norm;
    if (clip) {
      // a norm that is not finite would write NaN over every parameter of
      // the group: the group takes no step and its counter stands
      if (!isfinite(s.h)) c.skip = 1;
      else if (g.max_norm > 0.0) c.clip = (float)fmin(1.0, g.max_norm / (norm + 1e-6));
    }
  }
  if (!c.skip) groups[h].step = g.step + 1.0;
  c.beta1 = (float)g.beta1;
  c.one_m_beta1 = (float)(1.0 - g.beta1);
  c.beta2 = (float)g.beta2;
  c.one_m_beta2 = (float)(1.0 - g.beta2);
  c.decay = (float)(1.0 - g.lr * g.weight_decay);
  c.step_size = (float)g.lr / bc[0];
  c.rbc2 = 1.0f / sqrtf(bc[1]);
  c.eps = (float)g.eps;
  coef[h] = c;
}

// Chunks run last to first: the norm's pass read the gradients first to last,
// and the last of them are still in L2 (134M parameters with clipping: 653 ->
// 624 us for the call, 6.0 TB/s of what it cannot do without).  Parameters,
// gradients and moments are read before the wait for the coefficients: the
// kernel that makes those has itself waited for everything before it.
template <bool P16, bool G16>
__global__ void __launch_bounds__(kThreads)
    k_adamw32(const Chunk* __restrict__ chunks, const Coef* coef) {
  const Chunk t = chunks[gridDim.x - 1 - blockIdx.x];
  float p[4][4], g[4][4], m[4][4], v[4][4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = (u * kThreads + (int)threadIdx.x) * 4;
    load_n<G16, 4>(t.g, i, t.n, g[u]);
    load_n<P16, 4>(t.p, i, t.n, p[u]);
    load_n<false, 4>(t.m, i, t.n, m[u]);
    load_n<false, 4>(t.v, i, t.n, v[u]);
  }
  pdl_wait();
  pdl_launch_dependents();
  const Coef c = coef[t.group];
  if (c.skip) return;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = (u * kThreads + (int)threadIdx.x) * 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) (void)adamw1<false>(p[u][k], g[u][k], m[u][k], v[u][k], c);
    store_n<P16, 4>(t.p, i, t.n, p[u]);
    store_n<false, 4>(t.m, i, t.n, m[u]);
    store_n<false, 4>(t.v, i, t.n, v[u]);
  }
}

// Largest of a warp's non-negative values, as bit patterns (which order like
// the values, NaN above all: a block's scale then says it).
WS_DEVINL float warp_max_bits(uint32_t x) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, x));
}

// Codes of 8 values with their block's scale (ROOT: of roots, >= 0).  ANY: the
// scale may be subnormal, a few units of 2^-149 and rounded to one of them, so
// that quotients reach 2 and their code has to be held to 255 (a step's roots
// begin at 2^-74.5, far above; the clamp is for values that a caller brings).
// The quotients are the correctly rounded ones (a code border is where x / scale
// says it is) from the block's one reciprocal and a residual each (Markstein,
// IBM J. Res. Dev. 34, 1990), with tiny scales moved away from subnormal
// reciprocals.
template <bool ROOT, bool ANY>
WS_DEVINL void encode8(const float (&x)[8], float scale, uint32_t (&o)[2]) {
  const float up = scale < 0x1p-64f ? 0x1p64f : 1.0f;
  const float d = scale * up, inv = scale > 0.0f ? 1.0f / d : 0.0f;  // (all zero: codes 0)
  auto root = [](float v) { return ANY ? min(root_code(v), 255u) : root_code(v); };
  float q[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float y = x[k] * up, q0 = y * inv;
    q[k] = fmaf(fmaf(-q0, d, y), inv, q0);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t a = 0u;
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const float q0 = q[4 * h + k], q1 = q[4 * h + k + 1];
      a += (ROOT ? root(q0) + root(q1) * 256u : e4m3x2(q0, q1)) << (8 * k);
    }
    o[h] = a;
  }
}
template <bool ROOT>
WS_DEVINL void decode8(const uint32_t (&w)[2], float scale, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    if constexpr (ROOT) {
      x[k] = root_value(__byte_perm(w[k >> 2], 0u, 0x4440u + (k & 3)));
      x[k + 1] = root_value(__byte_perm(w[k >> 2], 0u, 0x4441u + (k & 3)));
    } else {
      e4m3x2_to_f32((w[k >> 2] >> (8 * (k & 3))) & 0xffffu, x[k], x[k + 1]);
    }
    x[k] *= scale;
    x[k + 1] *= scale;
  }
}
// 8 codes of one lane (left: how many exist; may be <= 0).
WS_DEVINL void load_codes(const uint8_t* q, int left, uint32_t (&w)[2]) {
  w[0] = w[1] = 0u;
  if (left >= 8) {
    const uint2 a = *reinterpret_cast<const uint2*>(q);
    w[0] = a.x, w[1] = a.y;
    return;
  }
#pragma unroll
  for (int k = 0; k < 7; ++k)
    if (k < left) w[k >> 2] |= (uint32_t)q[k] << (8 * (k & 3));
}
WS_DEVINL void store_codes(uint8_t* q, int left, const uint32_t (&w)[2]) {
  if (left >= 8) {
    *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    return;
  }
#pragma unroll
  for (int k = 0; k < 7; ++k)
    if (k < left) q[k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
}

// One warp per block of 256, 8 elements per lane.  The step uses the moments
// before they are rounded to 8 bits; the scales stay fp32.  Four CTAs an SM (a
// few spilled registers cost less than the fourth CTA's loads give: 39M
// parameters with bf16 gradients 119 -> 111 us).  134M fp32 parameters: 332 us,
// 6.5 TB/s; it was 410 us with a division for every code and a table lookup
// ahead of every chunk's addresses.
template <bool P16, bool G16>
__global__ void __launch_bounds__(kThreads, 4)
    k_adamw8(const Chunk* __restrict__ chunks, const Coef* coef) {
  const int lane = (int)lane_id(), warp = (int)warp_id();
  constexpr int kPer = kChunk / (kBlock8 * (kThreads / 32));  // blocks of a warp
  const Chunk t = chunks[gridDim.x - 1 - blockIdx.x];
  float pa[kPer][8], ga[kPer][8], sc[kPer][2];
  uint32_t ma[kPer][2], va[kPer][2];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int blk = u * (kThreads / 32) + warp, i = blk * kBlock8 + lane * 8;
    const int left = min(8, t.n - i);  // elements of this lane (may be <= 0)
    load_n<G16, 8>(t.g, i, t.n, ga[u]);
    load_n<P16, 8>(t.p, i, t.n, pa[u]);
    load_codes(static_cast<uint8_t*>(t.m) + i, left, ma[u]);
    load_codes(static_cast<uint8_t*>(t.v) + i, left, va[u]);
    const bool in = blk * kBlock8 < t.n;
    sc[u][0] = in ? t.ms[blk] : 0.0f;
    sc[u][1] = in ? t.vs[blk] : 0.0f;
  }
  pdl_wait();
  pdl_launch_dependents();
  const Coef c = coef[t.group];
  if (c.skip) return;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int blk = u * (kThreads / 32) + warp, i = blk * kBlock8 + lane * 8;
    if (blk * kBlock8 >= t.n) return;  // warp-uniform
    const int left = min(8, t.n - i);
    float(&p)[8] = pa[u];
    float(&g)[8] = ga[u];
    float m[8], v[8];
    decode8<false>(ma[u], sc[u][0], m);
    decode8<true>(va[u], sc[u][1], v);
    uint32_t mx = 0u, vx = 0u;  // as bit patterns: NaN is above all
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = v[k] * v[k];
      v[k] = adamw1<true>(p[k], g[k], m[k], v[k], c);  // what is kept is the root
      mx = max(mx, __float_as_uint(m[k]) & 0x7fffffffu);
      vx = max(vx, __float_as_uint(v[k]));
    }
    const float sm = warp_max_bits(mx) * (1.0f / kMTop), sv = warp_max_bits(vx) * (1.0f / kVTop);
    uint32_t mo[2], vo[2];
    encode8<false, false>(m, sm, mo);
    encode8<true, false>(v, sv, vo);
    store_n<P16, 8>(t.p, i, t.n, p);
    store_codes(static_cast<uint8_t*>(t.m) + i, left, mo);
    store_codes(static_cast<uint8_t*>(t.v) + i, left, vo);
    if (lane == 0) {
      t.ms[blk] = sm;
      t.vs[blk] = sv;
    }
  }
}

// Conversion of 8-bit states to and from fp32 (one warp per block of 256).
template <bool ROOT>
__global__ void __launch_bounds__(kThreads)
    k_adamw_encode8(const float* x, int64_t n, uint8_t* codes, float* scale) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t b = (int64_t)blockIdx.x * (kThreads / 32) + warp_id();
  if (b * kBlock8 >= n) return;
  const int i = (int)lane_id() * 8, nb = (int)min((int64_t)kBlock8, n - b * kBlock8);
  const int left = min(8, nb - i);
  float v[8];
  load_n<false, 8>(x + b * kBlock8, i, nb, v);
  uint32_t mx = 0u;
#pragma unroll
  for (int k = 0; k < 8; ++k) mx = max(mx, __float_as_uint(v[k]) & 0x7fffffffu);
  const float s = warp_max_bits(mx) * (ROOT ? 1.0f / kVTop : 1.0f / kMTop);
  uint32_t o[2];
  encode8<ROOT, true>(v, s, o);
  store_codes(codes + b * kBlock8 + i, left, o);
  if (lane_id() == 0) scale[b] = s;
}
template <bool ROOT, bool O16>
__global__ void __launch_bounds__(kThreads)
    k_adamw_decode8(const uint8_t* codes, const float* scale, int64_t n, void* out) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t b = (int64_t)blockIdx.x * (kThreads / 32) + warp_id();
  if (b * kBlock8 >= n) return;
  const int i = (int)lane_id() * 8, nb = (int)min((int64_t)kBlock8, n - b * kBlock8);
  uint32_t w[2];
  load_codes(codes + b * kBlock8 + i, min(8, nb - i), w);
  float v[8];
  decode8<ROOT>(w, scale[b], v);
  store_n<O16, 8>(static_cast<uint8_t*>(out) + b * kBlock8 * (O16 ? 2 : 4), i, nb, v);
}

bool al16p(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int64_t chunks_of(int64_t n) { return (n + kChunk - 1) / kChunk; }

// Checks of everything a plan is made of but overlaps.
ws_status check_tensors(const ws_adamw_tensor* t, int32_t n_tensors, int32_t n_groups,
                        const ws_adamw_types& ty, int64_t* n_chunks) {
  if (!t) return WS_ERR_INVALID;
  if (n_tensors < 1 || n_groups < 1 || n_groups > 65535) return WS_ERR_SHAPE;
  auto dt = [](int32_t d) { return d == WS_DTYPE_BF16 || d == WS_DTYPE_F32; };
  if (!dt(ty.p_dtype) || !dt(ty.g_dtype) || (ty.state_bits != 8 && ty.state_bits != 32))
    return WS_ERR_INVALID;
  int64_t c = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    if (!t[i].p || !t[i].g || !t[i].m || !t[i].v) return WS_ERR_INVALID;
    if (ty.state_bits == 8 && (!t[i].m_scale || !t[i].v_scale)) return WS_ERR_INVALID;
    if (t[i].group < 0 || t[i].group >= n_groups) return WS_ERR_INVALID;
    if (t[i].n < 1) return WS_ERR_SHAPE;
    if (!al16p(t[i].p) || !al16p(t[i].g) || !al16p(t[i].m) || !al16p(t[i].v)) return WS_ERR_ALIGN;
    if (ty.state_bits == 8 && ((reinterpret_cast<uintptr_t>(t[i].m_scale) | reinterpret_cast<uintptr_t>(t[i].v_scale)) & 3u))
      return WS_ERR_ALIGN;
    if (t[i].n > (int64_t)kChunk * 0x7fffffffll) return WS_ERR_SHAPE;
    c += chunks_of(t[i].n);
    if (c > 0x7fffffffll) return WS_ERR_SHAPE;
  }
  *n_chunks = c;
  return WS_OK;
}

}  // namespace

}  // namespace ws

using namespace ws;

extern "C" {

ws_status ws_adamw_plan_size(const ws_adamw_tensor* tensors, int32_t n_tensors, int32_t n_groups,
                             ws_adamw_types types, size_t* plan_bytes, size_t* workspace_bytes) {
  if (!plan_bytes || !workspace_bytes) return WS_ERR_INVALID;
  int64_t nc = 0;
  const ws_status s = check_tensors(tensors, n_tensors, n_groups, types, &nc);
  if (s != WS_OK) return s;
  *plan_bytes = plan_layout(n_groups, nc).bytes;
  *workspace_bytes = coef_bytes(n_groups) + (size_t)nc * sizeof(float2);
  return WS_OK;
}

ws_status ws_adamw_plan_init(const ws_adamw_tensor* tensors, int32_t n_tensors, int32_t n_groups,
                             ws_adamw_types types, void* image, size_t image_bytes,
                             ws_adamw_plan* plan) {
  if (!image || !plan) return WS_ERR_INVALID;
  int64_t nc = 0;
  const ws_status s = check_tensors(tensors, n_tensors, n_groups, types, &nc);
  if (s != WS_OK) return s;
  const Layout L = plan_layout(n_groups, nc);
  if (image_bytes < L.bytes) return WS_ERR_OOM;
  try {
    // every range the step writes, and the gradients, must be apart
    struct Range {
      uintptr_t b, e;
      bool grad;
    };
    std::vector<Range> r;
    r.reserve((size_t)n_tensors * 6);
    for (int32_t i = 0; i < n_tensors; ++i) {
      const ws_adamw_tensor& t = tensors[i];
      auto add = [&](const void* p, size_t bytes, bool grad) {
        r.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes, grad});
      };
      const size_t n = (size_t)t.n, st = types.state_bits == 8 ? n : n * 4;
      add(t.p, n * (types.p_dtype == WS_DTYPE_F32 ? 4 : 2), false);
      add(t.g, n * (types.g_dtype == WS_DTYPE_F32 ? 4 : 2), true);
      add(t.m, st, false);
      add(t.v, st, false);
      if (types.state_bits == 8) {
        const size_t sc = (n + kBlock8 - 1) / kBlock8 * 4;
        add(t.m_scale, sc, false);
        add(t.v_scale, sc, false);
      }
    }
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.b < b.b; });
    uintptr_t end_any = 0, end_written = 0;
    for (const Range& q : r) {
      // two gradients may be the same memory; nothing written may meet anything
      if (q.b < (q.grad ? end_written : end_any)) return WS_ERR_INVALID;
      end_any = std::max(end_any, q.e);
      if (!q.grad) end_written = std::max(end_written, q.e);
    }
  } catch (...) {  // no memory
    return WS_ERR_OOM;
  }
  memset(image, 0, L.bytes);
  uint8_t* im = static_cast<uint8_t*>(image);
  Chunk* ch = reinterpret_cast<Chunk*>(im + L.chunk);
  int32_t* gf = reinterpret_cast<int32_t*>(im + L.group_first);
  // chunks listed by group, tensors in the caller's order inside a group
  // (one pass over the tensors per group would be quadratic: count, then place)
  for (int32_t i = 0; i < n_tensors; ++i) gf[tensors[i].group + 1] += (int32_t)chunks_of(tensors[i].n);
  for (int32_t h = 0; h < n_groups; ++h) gf[h + 1] += gf[h];
  const int64_t pb = types.p_dtype == WS_DTYPE_F32 ? 4 : 2, gb = types.g_dtype == WS_DTYPE_F32 ? 4 : 2;
  const int64_t sb = types.state_bits / 8;
  for (int32_t i = 0; i < n_tensors; ++i) {
    const ws_adamw_tensor& t = tensors[i];
    for (int64_t e = 0; e < t.n; e += kChunk) {
      Chunk& c = ch[gf[t.group]++];
      c.p = static_cast<uint8_t*>(t.p) + e * pb;
      c.g = static_cast<const uint8_t*>(t.g) + e * gb;
      c.m = static_cast<uint8_t*>(t.m) + e * sb;
      c.v = static_cast<uint8_t*>(t.v) + e * sb;
      if (types.state_bits == 8) {
        c.ms = t.m_scale + e / kBlock8;
        c.vs = t.v_scale + e / kBlock8;
      }
      c.n = (int32_t)std::min<int64_t>(kChunk, t.n - e);
      c.group = t.group;
    }
  }
  // gf[h] now holds the end of group h: shift it back to the starts
  for (int32_t h = n_groups; h > 0; --h) gf[h] = gf[h - 1];
  gf[0] = 0;
  plan->image = nullptr;
  plan->types = types;
  plan->n_tensors = n_tensors;
  plan->n_groups = n_groups;
  plan->n_chunks = (int32_t)nc;
  return WS_OK;
}

ws_status ws_adamw_step(const ws_adamw_plan* plan, ws_adamw_group* groups, int32_t flags,
                        float* norms, void* workspace, size_t ws_bytes, ws_stream_t stream) {
  if (!plan || !plan->image || !groups || !workspace) return WS_ERR_INVALID;
  if (flags & ~WS_ADAMW_CLIP) return WS_ERR_INVALID;
  if (plan->n_tensors < 1 || plan->n_groups < 1 || plan->n_chunks < 1) return WS_ERR_INVALID;
  const ws_adamw_types ty = plan->types;
  auto dt = [](int32_t d) { return d == WS_DTYPE_BF16 || d == WS_DTYPE_F32; };
  if (!dt(ty.p_dtype) || !dt(ty.g_dtype) || (ty.state_bits != 8 && ty.state_bits != 32))
    return WS_ERR_INVALID;
  if (!al16p(plan->image) || !al16p(groups) || !al16p(workspace)) return WS_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(norms) & 3u) return WS_ERR_ALIGN;
  if (ws_bytes < coef_bytes(plan->n_groups) + (size_t)plan->n_chunks * sizeof(float2)) return WS_ERR_OOM;
  const Layout L = plan_layout(plan->n_groups, plan->n_chunks);
  const uint8_t* im = static_cast<const uint8_t*>(plan->image);
  const int32_t* gf = reinterpret_cast<const int32_t*>(im + L.group_first);
  const Chunk* ch = reinterpret_cast<const Chunk*>(im + L.chunk);
  Coef* coef = static_cast<Coef*>(workspace);
  float2* partial = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + coef_bytes(plan->n_groups));
  cudaStream_t st = (cudaStream_t)stream;
  const dim3 grid((unsigned)plan->n_chunks), block(kThreads);
  const bool p16 = ty.p_dtype == WS_DTYPE_BF16, g16 = ty.g_dtype == WS_DTYPE_BF16;
  const bool measure = (flags & WS_ADAMW_CLIP) || norms;
  cudaError_t e = cudaSuccess;
  if (measure) {
    note_launch();
    e = launch_pdl(g16 ? k_adamw_sumsq<true> : k_adamw_sumsq<false>,
                   dim3((unsigned)((plan->n_chunks + kSumChunks - 1) / kSumChunks)), block, 0, st, ch,
                   (int)plan->n_chunks, partial);
    if (e != cudaSuccess) return WS_ERR_CUDA;
  }
  note_launch();
  e = launch_pdl(k_adamw_begin, dim3((unsigned)plan->n_groups), dim3(kBeginThreads), 0, st, groups, gf,
                 (const float2*)(measure ? partial : nullptr), norms, (flags & WS_ADAMW_CLIP) ? 1 : 0, coef);
  if (e != cudaSuccess) return WS_ERR_CUDA;
  note_launch();
  void (*k)(const Chunk*, const Coef*);
  if (ty.state_bits == 32)
    k = p16 ? (g16 ? k_adamw32<true, true> : k_adamw32<true, false>)
            : (g16 ? k_adamw32<false, true> : k_adamw32<false, false>);
  else
    k = p16 ? (g16 ? k_adamw8<true, true> : k_adamw8<true, false>)
            : (g16 ? k_adamw8<false, true> : k_adamw8<false, false>);
  e = launch_pdl(k, grid, block, 0, st, ch, (const Coef*)coef);
  return e == cudaSuccess ? WS_OK : WS_ERR_CUDA;
}

namespace {
ws_status check_codes(const void* a, const void* codes, const float* scale, int64_t n, int32_t moment) {
  if (!a || !codes || !scale || (moment != WS_ADAMW_M && moment != WS_ADAMW_V_ROOT)) return WS_ERR_INVALID;
  if (n < 1 || n > (int64_t)kBlock8 * (kThreads / 32) * 0x7fffffffll) return WS_ERR_SHAPE;
  if (!al16p(a) || !al16p(codes) || (reinterpret_cast<uintptr_t>(scale) & 3u)) return WS_ERR_ALIGN;
  return WS_OK;
}
dim3 code_grid(int64_t n) {
  const int64_t per = (int64_t)kBlock8 * (kThreads / 32);
  return dim3((unsigned)((n + per - 1) / per));
}
}  // namespace

ws_status ws_adamw_encode8(const float* values, int64_t n, int32_t moment, uint8_t* codes,
                           float* scale, ws_stream_t stream) {
  const ws_status s = check_codes(values, codes, scale, n, moment);
  if (s != WS_OK) return s;
  note_launch();
  const cudaError_t e = launch_pdl(moment == WS_ADAMW_M ? k_adamw_encode8<false> : k_adamw_encode8<true>,
                                   code_grid(n), dim3(kThreads), 0, (cudaStream_t)stream, values, n, codes, scale);
  return e == cudaSuccess ? WS_OK : WS_ERR_CUDA;
}

ws_status ws_adamw_decode8(const uint8_t* codes, const float* scale, int64_t n, int32_t moment,
                           void* out, int32_t out_dtype, ws_stream_t stream) {
  const ws_status s = check_codes(out, codes, scale, n, moment);
  if (s != WS_OK) return s;
  if (out_dtype != WS_DTYPE_F32 && out_dtype != WS_DTYPE_BF16) return WS_ERR_INVALID;
  const bool o16 = out_dtype == WS_DTYPE_BF16;
  note_launch();
  const cudaError_t e =
      launch_pdl(moment == WS_ADAMW_M ? (o16 ? k_adamw_decode8<false, true> : k_adamw_decode8<false, false>)
                                      : (o16 ? k_adamw_decode8<true, true> : k_adamw_decode8<true, false>),
                 code_grid(n), dim3(kThreads), 0, (cudaStream_t)stream, codes, scale, n, out);
  return e == cudaSuccess ? WS_OK : WS_ERR_CUDA;
}

}  // extern "C"
