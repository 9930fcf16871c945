// adamw.cu -- one AdamW step over many tensors (decoupled weight decay,
// Loshchilov & Hutter, 2019), moments in 32 bits or in 8, with the global
// gradient norm of each parameter group and clipping by it.
//
// All tensors of a plan run in one launch: the plan cuts every tensor into
// chunks of kChunk elements and lists the chunks by group, so CTA c reads
// which tensor it works on from the chunk table.  Every operand is read once
// and written once; each element needs the group's coefficients only, so the
// step is bound by memory (28 bytes per fp32 parameter with 32-bit states,
// 16 with 8-bit ones).
//
// Sums of squares run in a fixed order (inside a thread, a fixed butterfly in
// the warp, warps and then chunks in index order, the chunks' sums in double),
// so a norm does not depend on the launch.
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

// Device image of one tensor of a plan (64 bytes).
struct TensorDev {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t n;
  int32_t group;
  int32_t first_chunk;  // index of the tensor's first chunk in the table
};
static_assert(sizeof(TensorDev) == 64, "tensor entry");

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

// Sections of the plan image and of the workspace.
struct Layout {
  size_t tensors, group_first, chunk, bytes;  // plan: entries, first chunk of each group, chunk -> tensor
};
Layout plan_layout(int32_t n_tensors, int32_t n_groups, int64_t n_chunks) {
  Layout L{};
  L.tensors = 0;
  L.group_first = al16((size_t)n_tensors * sizeof(TensorDev));
  L.chunk = L.group_first + al16((size_t)(n_groups + 1) * 4);
  L.bytes = L.chunk + al16((size_t)n_chunks * 4);
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
  const uint32_t b = __float_as_uint(q);
  const uint32_t r = (b + 0x3FFFFu + ((b >> 19) & 1u)) >> 19;
  const int c = max(1, min(255, (int)r - (int)kRootBias));
  return q > 0.0f ? (uint32_t)c : 0u;
}
WS_DEVINL float root_value(uint32_t c) {
  return c ? __uint_as_float((c + kRootBias) << 19) : 0.0f;
}
constexpr float kMTop = 448.0f, kVTop = 1.9375f;

// ---- elements ------------------------------------------------------------------------
// N (4 or 8) consecutive elements from i0 of an fp32 or bf16 array of n; past
// the end they read as 0 and are not written.  Full vectors use 16-byte (bf16
// x 4: 8-byte) accesses.
template <bool BF16, int N>
WS_DEVINL void load_n(const void* base, int64_t i0, int64_t n, float (&x)[N]) {
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
WS_DEVINL void store_n(void* base, int64_t i0, int64_t n, const float (&x)[N]) {
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

// m, v and p of one element.  Products and sums are rounded one by one (no
// contraction), as the formula is written: a value that lies on the border
// between two 8-bit codes then falls the way it does for anybody who
// evaluates the formula in fp32.
WS_DEVINL void adamw1(float& p, float g, float& m, float& v, const Coef& c) {
  g = __fmul_rn(g, c.clip);
  m = __fadd_rn(__fmul_rn(m, c.beta1), __fmul_rn(g, c.one_m_beta1));
  v = __fadd_rn(__fmul_rn(v, c.beta2), __fmul_rn(__fmul_rn(g, g), c.one_m_beta2));
  const float den = fmaf(sqrtf(v), c.rbc2, c.eps);
  p = p * c.decay - c.step_size * (m / den);
}

// ---- kernels ---------------------------------------------------------------------------
template <bool G16>
__global__ void __launch_bounds__(kThreads)
    k_adamw_sumsq(const TensorDev* __restrict__ tensors, const int32_t* __restrict__ chunk,
                  double* __restrict__ partial) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float red[kThreads / 32];
  const TensorDev t = tensors[chunk[blockIdx.x]];
  const int64_t base = (int64_t)((int)blockIdx.x - t.first_chunk) * kChunk;
  float g[4][4];
#pragma unroll
  for (int u = 0; u < 4; ++u) load_n<G16, 4>(t.g, base + (u * kThreads + threadIdx.x) * 4, t.n, g[u]);
  float s = 0.0f;
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int k = 0; k < 4; ++k) s = fmaf(g[u][k], g[u][k], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane_id() == 0) red[warp_id()] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double d = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) d += (double)red[w];
    partial[blockIdx.x] = d;
  }
}

// One CTA per group: the norm from the chunks' sums (double, chunk order per
// thread, threads in index order), the step counter and the coefficients.
__global__ void __launch_bounds__(kThreads)
    k_adamw_begin(ws_adamw_group* __restrict__ groups, const int32_t* __restrict__ group_first,
                  const double* __restrict__ partial, float* __restrict__ norms, int clip,
                  Coef* __restrict__ coef) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ double red[kThreads / 32];
  const int h = blockIdx.x;
  double norm = 0.0;
  if (partial) {
    double s = 0.0;
    for (int i = group_first[h] + threadIdx.x; i < group_first[h + 1]; i += kThreads) s += partial[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane_id() == 0) red[warp_id()] = s;
    __syncthreads();
    if (threadIdx.x == 0)
      for (int w = 0; w < kThreads / 32; ++w) norm += red[w];
    norm = sqrt(norm);
  }
  if (threadIdx.x != 0) return;
  ws_adamw_group g = groups[h];
  Coef c{};
  c.clip = 1.0f;
  if (partial) {
    if (norms) norms[h] = (float)norm;
    if (clip) {
      // a norm that is not finite would write NaN over every parameter of
      // the group: the group takes no step and its counter stands
      if (!isfinite(norm)) c.skip = 1;
      else if (g.max_norm > 0.0) c.clip = (float)fmin(1.0, g.max_norm / (norm + 1e-6));
    }
  }
  if (!c.skip) {
    g.step += 1.0;
    groups[h].step = g.step;
  }
  c.beta1 = (float)g.beta1;
  c.one_m_beta1 = (float)(1.0 - g.beta1);
  c.beta2 = (float)g.beta2;
  c.one_m_beta2 = (float)(1.0 - g.beta2);
  c.decay = (float)(1.0 - g.lr * g.weight_decay);
  c.step_size = (float)(g.lr / (1.0 - pow(g.beta1, g.step)));
  c.rbc2 = (float)(1.0 / sqrt(1.0 - pow(g.beta2, g.step)));
  c.eps = (float)g.eps;
  coef[h] = c;
}

template <bool P16, bool G16>
__global__ void __launch_bounds__(kThreads)
    k_adamw32(const TensorDev* __restrict__ tensors, const int32_t* __restrict__ chunk,
              const Coef* __restrict__ coef) {
  pdl_wait();
  pdl_launch_dependents();
  const TensorDev t = tensors[chunk[blockIdx.x]];
  const Coef c = coef[t.group];
  if (c.skip) return;
  const int64_t base = (int64_t)((int)blockIdx.x - t.first_chunk) * kChunk;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t i = base + (u * kThreads + threadIdx.x) * 4;
    float p[4], g[4], m[4], v[4];
    load_n<P16, 4>(t.p, i, t.n, p);
    load_n<G16, 4>(t.g, i, t.n, g);
    load_n<false, 4>(t.m, i, t.n, m);
    load_n<false, 4>(t.v, i, t.n, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) adamw1(p[k], g[k], m[k], v[k], c);
    store_n<P16, 4>(t.p, i, t.n, p);
    store_n<false, 4>(t.m, i, t.n, m);
    store_n<false, 4>(t.v, i, t.n, v);
  }
}

// Larger of two values; NaN wins and stays, so that a block's scale says it.
WS_DEVINL float max_nan(float a, float b) { return (b > a || b != b) ? b : a; }
// Largest of a warp's non-negative values, NaN above all (as bit patterns
// they order like integers).
WS_DEVINL float warp_max_nonneg(float x) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x) & 0x7fffffffu));
}

// Codes of 8 values with their block's scale (ROOT: of roots, >= 0).
template <bool ROOT>
WS_DEVINL void encode8(const float (&x)[8], float scale, uint32_t (&o)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t a = 0u;
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const int e = 4 * h + k;
      const float q0 = scale > 0.0f ? x[e] / scale : 0.0f, q1 = scale > 0.0f ? x[e + 1] / scale : 0.0f;
      a |= (ROOT ? root_code(q0) | (root_code(q1) << 8) : e4m3x2(q0, q1)) << (8 * k);
    }
    o[h] = a;
  }
}
template <bool ROOT>
WS_DEVINL void decode8(const uint32_t (&w)[2], float scale, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const uint32_t c = w[k >> 2] >> (8 * (k & 3));
    if constexpr (ROOT) {
      x[k] = root_value(c & 255u);
      x[k + 1] = root_value((c >> 8) & 255u);
    } else {
      e4m3x2_to_f32(c & 0xffffu, x[k], x[k + 1]);
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
// before they are rounded to 8 bits; the scales stay fp32.
template <bool P16, bool G16>
__global__ void __launch_bounds__(kThreads)
    k_adamw8(const TensorDev* __restrict__ tensors, const int32_t* __restrict__ chunk,
             const Coef* __restrict__ coef) {
  pdl_wait();
  pdl_launch_dependents();
  const TensorDev t = tensors[chunk[blockIdx.x]];
  const Coef c = coef[t.group];
  if (c.skip) return;
  const int64_t base = (int64_t)((int)blockIdx.x - t.first_chunk) * kChunk;
  const int lane = (int)lane_id();
#pragma unroll
  for (int u = 0; u < kChunk / (kBlock8 * (kThreads / 32)); ++u) {
    const int64_t b0 = base + (int64_t)(u * (kThreads / 32) + (int)warp_id()) * kBlock8;
    if (b0 >= t.n) return;  // warp-uniform
    const int64_t i = b0 + lane * 8;
    const int left = (int)min((int64_t)8, t.n - i);  // elements of this lane (may be <= 0)
    float p[8], g[8], m[8], v[8];
    load_n<P16, 8>(t.p, i, t.n, p);
    load_n<G16, 8>(t.g, i, t.n, g);
    uint8_t* mq = static_cast<uint8_t*>(t.m) + i;
    uint8_t* vq = static_cast<uint8_t*>(t.v) + i;
    uint32_t mw[2], vw[2];
    load_codes(mq, left, mw);
    load_codes(vq, left, vw);
    decode8<false>(mw, t.ms[b0 / kBlock8], m);
    decode8<true>(vw, t.vs[b0 / kBlock8], v);
    float mx = 0.0f, vx = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = v[k] * v[k];
      adamw1(p[k], g[k], m[k], v[k], c);
      v[k] = sqrtf(v[k]);  // what is kept is the root
      mx = max_nan(mx, fabsf(m[k]));
      vx = max_nan(vx, v[k]);
    }
    const float sm = warp_max_nonneg(mx) / kMTop, sv = warp_max_nonneg(vx) / kVTop;
    uint32_t mo[2], vo[2];
    encode8<false>(m, sm, mo);
    encode8<true>(v, sv, vo);
    store_n<P16, 8>(t.p, i, t.n, p);
    store_codes(mq, left, mo);
    store_codes(vq, left, vo);
    if (lane == 0) {
      t.ms[b0 / kBlock8] = sm;
      t.vs[b0 / kBlock8] = sv;
    }
  }
}

// Conversion of 8-bit states to and from fp32 (one warp per block of 256).
template <bool ROOT>
__global__ void __launch_bounds__(kThreads)
    k_adamw_encode8(const float* __restrict__ x, int64_t n, uint8_t* __restrict__ codes,
                    float* __restrict__ scale) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t b = (int64_t)blockIdx.x * (kThreads / 32) + warp_id();
  if (b * kBlock8 >= n) return;
  const int64_t i = b * kBlock8 + lane_id() * 8;
  const int left = (int)min((int64_t)8, n - i);
  float v[8];
  load_n<false, 8>(x, i, n, v);
  float mx = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) mx = max_nan(mx, fabsf(v[k]));
  const float s = warp_max_nonneg(mx) / (ROOT ? kVTop : kMTop);
  uint32_t o[2];
  encode8<ROOT>(v, s, o);
  store_codes(codes + i, left, o);
  if (lane_id() == 0) scale[b] = s;
}
template <bool ROOT, bool O16>
__global__ void __launch_bounds__(kThreads)
    k_adamw_decode8(const uint8_t* __restrict__ codes, const float* __restrict__ scale, int64_t n,
                    void* __restrict__ out) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t b = (int64_t)blockIdx.x * (kThreads / 32) + warp_id();
  if (b * kBlock8 >= n) return;
  const int64_t i = b * kBlock8 + lane_id() * 8;
  uint32_t w[2];
  load_codes(codes + i, (int)min((int64_t)8, n - i), w);
  float v[8];
  decode8<ROOT>(w, scale[b], v);
  store_n<O16, 8>(out, i, n, v);
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
  *plan_bytes = plan_layout(n_tensors, n_groups, nc).bytes;
  *workspace_bytes = coef_bytes(n_groups) + (size_t)nc * sizeof(double);
  return WS_OK;
}

ws_status ws_adamw_plan_init(const ws_adamw_tensor* tensors, int32_t n_tensors, int32_t n_groups,
                             ws_adamw_types types, void* image, size_t image_bytes,
                             ws_adamw_plan* plan) {
  if (!image || !plan) return WS_ERR_INVALID;
  int64_t nc = 0;
  const ws_status s = check_tensors(tensors, n_tensors, n_groups, types, &nc);
  if (s != WS_OK) return s;
  const Layout L = plan_layout(n_tensors, n_groups, nc);
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
  } catch (const std::bad_alloc&) {
    return WS_ERR_OOM;
  }
  memset(image, 0, L.bytes);
  uint8_t* im = static_cast<uint8_t*>(image);
  TensorDev* td = reinterpret_cast<TensorDev*>(im + L.tensors);
  int32_t* gf = reinterpret_cast<int32_t*>(im + L.group_first);
  int32_t* ch = reinterpret_cast<int32_t*>(im + L.chunk);
  // chunks listed by group, tensors in the caller's order inside a group
  // (one pass over the tensors per group would be quadratic: count, then place)
  for (int32_t i = 0; i < n_tensors; ++i) gf[tensors[i].group + 1] += (int32_t)chunks_of(tensors[i].n);
  for (int32_t h = 0; h < n_groups; ++h) gf[h + 1] += gf[h];
  for (int32_t i = 0; i < n_tensors; ++i) {
    const ws_adamw_tensor& t = tensors[i];
    const int32_t first = gf[t.group], c = (int32_t)chunks_of(t.n);
    td[i] = TensorDev{t.p, t.g, t.m, t.v, t.m_scale, t.v_scale, t.n, t.group, first};
    for (int32_t k = 0; k < c; ++k) ch[first + k] = i;
    gf[t.group] = first + c;
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
  if (ws_bytes < coef_bytes(plan->n_groups) + (size_t)plan->n_chunks * sizeof(double)) return WS_ERR_OOM;
  const Layout L = plan_layout(plan->n_tensors, plan->n_groups, plan->n_chunks);
  const uint8_t* im = static_cast<const uint8_t*>(plan->image);
  const TensorDev* td = reinterpret_cast<const TensorDev*>(im + L.tensors);
  const int32_t* gf = reinterpret_cast<const int32_t*>(im + L.group_first);
  const int32_t* ch = reinterpret_cast<const int32_t*>(im + L.chunk);
  Coef* coef = static_cast<Coef*>(workspace);
  double* partial = reinterpret_cast<double*>(static_cast<uint8_t*>(workspace) + coef_bytes(plan->n_groups));
  cudaStream_t st = (cudaStream_t)stream;
  const dim3 grid((unsigned)plan->n_chunks), block(kThreads);
  const bool p16 = ty.p_dtype == WS_DTYPE_BF16, g16 = ty.g_dtype == WS_DTYPE_BF16;
  const bool measure = (flags & WS_ADAMW_CLIP) || norms;
  cudaError_t e = cudaSuccess;
  if (measure) {
    note_launch();
    e = launch_pdl(g16 ? k_adamw_sumsq<true> : k_adamw_sumsq<false>, grid, block, 0, st, td, ch, partial);
    if (e != cudaSuccess) return WS_ERR_CUDA;
  }
  note_launch();
  e = launch_pdl(k_adamw_begin, dim3((unsigned)plan->n_groups), block, 0, st, groups, gf,
                 (const double*)(measure ? partial : nullptr), norms, (flags & WS_ADAMW_CLIP) ? 1 : 0, coef);
  if (e != cudaSuccess) return WS_ERR_CUDA;
  note_launch();
  void (*k)(const TensorDev*, const int32_t*, const Coef*);
  if (ty.state_bits == 32)
    k = p16 ? (g16 ? k_adamw32<true, true> : k_adamw32<true, false>)
            : (g16 ? k_adamw32<false, true> : k_adamw32<false, false>);
  else
    k = p16 ? (g16 ? k_adamw8<true, true> : k_adamw8<true, false>)
            : (g16 ? k_adamw8<false, true> : k_adamw8<false, false>);
  e = launch_pdl(k, grid, block, 0, st, td, ch, (const Coef*)coef);
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
