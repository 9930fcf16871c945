// rope.cu -- the step between the q and k projections and the attention core:
// RMS norm of each head with a gain, then rotary positions (Su et al., 2021),
// in one pass over the rows, and its backward pass.
//
//   n = x / sqrt(mean(x^2) + eps) * gain           over one head's elements
//   (y_a, y_b) = c (n_a cos t - n_b sin t, n_a sin t + n_b cos t)
// for the pairs (a, b) of the head's first rot elements: (i, i + rot/2), or
// interleaved (2i, 2i + 1).  The angle of pair i at position p is p times a
// frequency.  The frequencies come as 64-bit fractions of a turn, so p times
// one, modulo 2^64, is the fraction of a turn exactly, however far the
// position: the angle's error is fp32's, not the position's.
//
// Backward, with d the upstream gradient rotated back, u = x / sqrt(...):
//   dgain = sum d u,   dx = (d gain - u mean(d gain u)) / sqrt(...)
//
// What bounds it: memory (4 bytes an element forward, 6 backward).  A group of
// D/16 threads has one token and walks over some of its heads, so the sines
// and cosines (eight pairs a thread, in registers) serve all of them; a thread
// has both elements of each of its pairs, two 16-byte pieces a head, and the
// only exchange is the head's sum.  16384 rows of 40 + 8 heads of 128 take 71 us
// (5.7 TB/s), 8192 rows of 28 + 4 backward 38 us (5.3 TB/s).
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace ws {
namespace {

constexpr int kRopeThreads = 256;
// Heads a group has in flight at a time.  16384 tokens of 40 + 8 heads: 92 us with
// two, 77 with four, 72 with eight; backward (two inputs a head, and registers for
// the gains' gradients), 8192 tokens of 28 + 4: 52 with one, 39.5 with two, 54 with
// three.
constexpr int kFwdBatch = 8;
constexpr int kBwdBatch = 2;
constexpr int kGainRow = kRopeThreads + 8;  // floats of a row of the threads' sums, padded
constexpr int kGainRows = 32;    // rows that k_rope_gain adds side by side

struct RopeArgs {
  const uint64_t* turns;  // [rot/2] 2^-64 turns a position; NULL: no rotation
  const int32_t* pos;     // [M]
  const float *gq, *gk;   // [D] or NULL: no norm
  const uint16_t *q, *k;  // inputs of the forward
  const uint16_t *uq, *uk;  // backward: upstream gradients
  uint16_t *oq, *ok;      // outputs
  int64_t sq, sk, suq, suk, soq, sok;  // row strides in elements
  float* partial;         // backward with gradients of the gains: [CTAs][2][D]
  int64_t M;
  int rot, nh, nkv, parts;  // a token's heads are dealt to `parts` groups
  float factor, eps;
};

struct Vec16 {
  float v[16];  // two pieces of eight elements
};
WS_DEVINL void load16(const uint16_t* p, int c0, int c1, uint4 (&r)[2]) {
  r[0] = *reinterpret_cast<const uint4*>(p + c0 * 8);
  r[1] = *reinterpret_cast<const uint4*>(p + c1 * 8);
}
WS_DEVINL Vec16 unpack16(const uint4 (&r)[2]) {
  Vec16 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o.v[8 * i + 2 * j] = bf16_lo(w[j]);
      o.v[8 * i + 2 * j + 1] = bf16_hi(w[j]);
    }
  }
  return o;
}
WS_DEVINL void store16(uint16_t* p, int c0, int c1, const Vec16& o) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint4 w;
    w.x = pack_bf16x2(o.v[8 * i], o.v[8 * i + 1]);
    w.y = pack_bf16x2(o.v[8 * i + 2], o.v[8 * i + 3]);
    w.z = pack_bf16x2(o.v[8 * i + 4], o.v[8 * i + 5]);
    w.w = pack_bf16x2(o.v[8 * i + 6], o.v[8 * i + 7]);
    *reinterpret_cast<uint4*>(p + (i ? c1 : c0) * 8) = w;
  }
}
// Sum over the T threads of a group (every thread of the warp takes part).
template <int T>
WS_DEVINL float group_sum(float x) {
#pragma unroll
  for (int o = T / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// The thread's pairs turned by their angles (sign = 1) or back (-1).
template <bool IL>
WS_DEVINL void turn(Vec16& x, const float (&cs)[8], const float (&sn)[8], float sign) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int a = IL ? 2 * j : j, b = IL ? 2 * j + 1 : j + 8;
    const float s = sign * sn[j], xa = x.v[a], xb = x.v[b];
    x.v[a] = xa * cs[j] - xb * s;
    x.v[b] = xa * s + xb * cs[j];
  }
}

// What a group's threads know of their token: pieces, angles.
template <int D, bool IL>
struct Token {
  int c0, c1;
  bool rotates;
  float cs[8], sn[8];
  WS_DEVINL Token(const RopeArgs& a, int t, int64_t m) {
    const int rt = a.turns ? a.rot / 16 : 0;  // threads whose elements are rotated
    rotates = t < rt;
    c0 = rotates ? t : 2 * t;
    c1 = rotates ? t + rt : 2 * t + 1;
    if (!rotates) return;
    const uint64_t p = (uint64_t)(int64_t)a.pos[m];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = !IL ? 8 * t + j : j < 4 ? 4 * t + j : 4 * (t + rt) + j - 4;
      // the top 32 bits of the fraction, as half turns in [-1, 1)
      const float half = (float)(int32_t)((p * a.turns[i]) >> 32) * 0x1p-31f;
      float s, c;
      sincospif(half, &s, &c);
      cs[j] = c * a.factor;
      sn[j] = s * a.factor;
    }
  }
};

WS_DEVINL void load_gain(const float* g, int c0, int c1, float (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = *reinterpret_cast<const float4*>(g + (i < 2 ? c0 : c1) * 8 + (i & 1) * 4);
    w[4 * i] = f.x;
    w[4 * i + 1] = f.y;
    w[4 * i + 2] = f.z;
    w[4 * i + 3] = f.w;
  }
}

// Heads part, part + parts, ... of one input of one token.
template <int D, bool IL>
WS_DEVINL void fwd_heads(const RopeArgs& a, const Token<D, IL>& tok, const uint16_t* x, uint16_t* o,
                         const float* gain, int first, int heads, bool live) {
  float w[16];
  if (gain) load_gain(gain, tok.c0, tok.c1, w);
  // a warp's groups have different tokens and parts but take the same steps:
  // one whose heads are through goes along with zeros
  for (int j0 = 0; j0 < heads; j0 += kFwdBatch * a.parts) {
    uint4 raw[kFwdBatch][2];
#pragma unroll
    for (int i = 0; i < kFwdBatch; ++i) {
      const int h = j0 + i * a.parts + first;
      if (h < heads)
        load16(x + h * D, tok.c0, tok.c1, raw[i]);
      else
        raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kFwdBatch; ++i) {
      if (j0 + i * a.parts >= heads) break;
      const int h = j0 + i * a.parts + first;
      Vec16 v = unpack16(raw[i]);
      if (gain) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) s += v.v[j] * v.v[j];
        const float r = rsqrtf(group_sum<D / 16>(s) * (1.0f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < 16; ++j) v.v[j] = v.v[j] * r * w[j];
      }
      if (tok.rotates) turn<IL>(v, tok.cs, tok.sn, 1.0f);
      if (live && h < heads) store16(o + h * D, tok.c0, tok.c1, v);
    }
  }
}

template <int D, bool IL>
__global__ void __launch_bounds__(kRopeThreads) k_rope_fwd(const RopeArgs a) {
  constexpr int T = D / 16;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t unit = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) / T;
  const bool live = unit < a.M * a.parts;
  const int64_t m = live ? unit / a.parts : 0;
  const int part = live ? (int)(unit % a.parts) : 0;
  const Token<D, IL> tok(a, (int)threadIdx.x % T, m);
  fwd_heads<D, IL>(a, tok, a.q + m * a.sq, a.oq + m * a.soq, a.gq, part, a.nh, live);
  // the deal goes on with the kv heads
  const int first = (part - a.nh % a.parts + a.parts) % a.parts;
  fwd_heads<D, IL>(a, tok, a.k + m * a.sk, a.ok + m * a.sok, a.gk, first, a.nkv, live);
}

template <int D, bool IL, bool GAINS>
WS_DEVINL void bwd_heads(const RopeArgs& a, const Token<D, IL>& tok, const uint16_t* x,
                         const uint16_t* u, uint16_t* o, const float* gain, int first, int heads,
                         bool live, float* sums) {
  constexpr int B = kBwdBatch;
  float dg[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) dg[j] = 0.0f;
  float w[16];
  if (gain) load_gain(gain, tok.c0, tok.c1, w);
  for (int j0 = 0; j0 < heads; j0 += B * a.parts) {
    uint4 rx[B][2], ru[B][2];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int h = j0 + i * a.parts + first;
      rx[i][0] = rx[i][1] = ru[i][0] = ru[i][1] = make_uint4(0, 0, 0, 0);
      if (h < heads) {
        load16(u + h * D, tok.c0, tok.c1, ru[i]);
        if (gain) load16(x + h * D, tok.c0, tok.c1, rx[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (j0 + i * a.parts >= heads) break;
      const int h = j0 + i * a.parts + first;
      Vec16 d = unpack16(ru[i]);
      if (tok.rotates) turn<IL>(d, tok.cs, tok.sn, -1.0f);
      if (gain) {
        Vec16 n = unpack16(rx[i]);
        float s = 0.0f, e = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          s += n.v[j] * n.v[j];
          e += d.v[j] * w[j] * n.v[j];
        }
        const float r = rsqrtf(group_sum<D / 16>(s) * (1.0f / D) + a.eps);
        e = group_sum<D / 16>(e) * r * (1.0f / D);  // mean(d gain u)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float uj = n.v[j] * r;
          if (GAINS && live && h < heads) dg[j] += d.v[j] * uj;
          d.v[j] = r * (d.v[j] * w[j] - uj * e);
        }
      }
      if (live && h < heads) store16(o + h * D, tok.c0, tok.c1, d);
    }
  }
  if (GAINS) {
#pragma unroll
    for (int j = 0; j < 16; ++j) sums[j * kGainRow] += dg[j];
  }
}

// The CTAs take the (token, part) units in turn.  A thread's share of the gains'
// gradients grows in its own place in shared memory, a unit's heads at a time; then
// the CTA's groups are summed in their order.  16384 tokens of 40 + 8 heads: 132 us
// (4.6 TB/s); with the sums of all units in registers, which leave one CTA an SM,
// 172.
template <int D, bool IL, bool GAINS>
__global__ void __launch_bounds__(kRopeThreads, 2) k_rope_bwd(const RopeArgs a) {
  constexpr int T = D / 16, G = kRopeThreads / T;
  __shared__ float sum[GAINS ? 32 : 1][kGainRow];  // [q, k][element of the thread][thread]
  pdl_wait();
  pdl_launch_dependents();
  const int tid = (int)threadIdx.x, t = tid % T, g = tid / T;
  const int64_t units = a.M * a.parts;
  if (GAINS)
    for (int j = 0; j < 32; ++j) sum[j][tid] = 0.0f;
  for (int64_t u0 = (int64_t)blockIdx.x * G; u0 < units; u0 += (int64_t)gridDim.x * G) {
    const int64_t unit = u0 + g;
    const bool live = unit < units;
    const int64_t m = live ? unit / a.parts : 0;
    const int part = live ? (int)(unit % a.parts) : 0;
    const Token<D, IL> tok(a, t, m);
    bwd_heads<D, IL, GAINS>(a, tok, a.q + m * a.sq, a.uq + m * a.suq, a.oq + m * a.soq, a.gq, part,
                            a.nh, live, &sum[0][tid]);
    const int first = (part - a.nh % a.parts + a.parts) % a.parts;
    bwd_heads<D, IL, GAINS>(a, tok, a.k + m * a.sk, a.uk + m * a.suk, a.ok + m * a.sok, a.gk, first,
                            a.nkv, live, &sum[GAINS ? 16 : 0][tid]);
  }
  if (GAINS) {
    __syncthreads();
    const int rt = a.turns ? a.rot / 16 : 0;
    for (int i = tid; i < 2 * D; i += kRopeThreads) {
      const int row = i / T, c = i % T, j = row & 15;  // element j of the groups' threads c
      float s = 0.0f;
      for (int k = 0; k < G; ++k) s += sum[row][k * T + c];
      const int piece = j < 8 ? (c < rt ? c : 2 * c) : (c < rt ? c + rt : 2 * c + 1);
      a.partial[((int64_t)blockIdx.x * 2 + (row >> 4)) * D + piece * 8 + (j & 7)] = s;
    }
  }
}

// Gradients of the gains from the CTAs' shares [n][2][D]: 32 columns a CTA,
// kGainRows rows side by side, joined in their order.
__global__ void __launch_bounds__(32 * kGainRows) k_rope_gain(const float* partial, int n, int D,
                                                              float* dgq, float* dgk, int accumulate) {
  __shared__ float sum[kGainRows][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = (int)threadIdx.x & 31, row = (int)threadIdx.x >> 5;
  const int col = (int)blockIdx.x * 32 + lane;  // of [2][D]
  float s = 0.0f;
  for (int i = row; i < n; i += kGainRows) s += partial[(int64_t)i * 2 * D + col];
  sum[row][lane] = s;
  __syncthreads();
  float* out = col < D ? dgq : dgk;
  if (row || !out) return;
  s = 0.0f;
  for (int i = 0; i < kGainRows; ++i) s += sum[i][lane];
  float* p = out + col % D;
  *p = accumulate ? *p + s : s;
}

bool al16r(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al4r(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

ws_status rope_shape(int64_t M, int32_t nh, int32_t nkv, int32_t hd) {
  if (M < 1 || M > (int64_t)1 << 30 || nh < 1 || nkv < 1 || nh > 1024 || nkv > 1024) return WS_ERR_SHAPE;
  return hd == 64 || hd == 128 ? WS_OK : WS_ERR_SHAPE;
}

// Threads of an SM whose groups a call is dealt to: about as many as it holds at
// the kernels' registers (with twice as many the backward of 512 tokens took 23 us
// for 17, that of 8192 tokens 45 for 39); for the backward with gradients of gains
// the two CTAs that run at once (2048 tokens of 40 + 8 heads: 22 us, with 768 and
// four CTAs 28.5, with 256 and two 28).
constexpr int kFullThreads = 768, kGainThreads = 512;
int64_t full_groups(int hd, int threads) { return (int64_t)device_sm_count() * threads / (hd / 16); }

// Groups a token's heads are dealt to: as few as fill the device (each then
// makes the sines and cosines for more heads).
int rope_parts(int64_t M, int heads, int hd, int threads = kFullThreads) {
  const int64_t want = full_groups(hd, threads) / M;
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, heads));
}
int64_t rope_ctas(int64_t M, int parts, int hd) {
  const int64_t g = kRopeThreads / (hd / 16);
  return (M * parts + g - 1) / g;
}
// CTAs of the backward where they sum gradients: no more than run at once.
int64_t rope_gain_ctas(int64_t M, int parts, int hd) {
  return std::min<int64_t>(rope_ctas(M, parts, hd), (int64_t)device_sm_count() * kGainThreads / kRopeThreads);
}

ws_status check_io(const void* p, int64_t stride, int32_t heads, int32_t hd) {
  if (!p) return WS_ERR_INVALID;
  if (stride < (int64_t)heads * hd || stride % 8 || stride > (int64_t)1 << 31) return WS_ERR_SHAPE;
  return al16r(p) ? WS_OK : WS_ERR_ALIGN;
}
// An output may be an input itself, row for row.
bool same_rows(const void* in, int64_t si, const void* out, int64_t so) { return in != out || si == so; }

ws_status check_rope(const ws_rope* r, const int32_t* pos, const float* gq, const float* gk, float eps,
                     int32_t hd) {
  if (!r && !gq && !gk) return WS_ERR_INVALID;
  if (r) {
    if (!r->turns || !pos || r->reserved || (r->interleaved & ~1)) return WS_ERR_INVALID;
    if (r->rot < 16 || r->rot > hd || r->rot % 16) return WS_ERR_SHAPE;
    if (!isfinite(r->factor)) return WS_ERR_INVALID;
    if (!al16r(r->turns) || !al4r(pos)) return WS_ERR_ALIGN;
  }
  if (!(eps >= 0.0f) || !isfinite(eps)) return WS_ERR_INVALID;
  if ((gq && !al16r(gq)) || (gk && !al16r(gk))) return WS_ERR_ALIGN;
  return WS_OK;
}

RopeArgs rope_args(const ws_rope* r, const int32_t* pos, int64_t M, int32_t nh, int32_t nkv, int32_t hd,
                   float eps, const float* gq, const float* gk) {
  RopeArgs a = {};
  a.turns = r ? r->turns : nullptr;
  a.rot = r ? r->rot : 0;
  a.factor = r ? r->factor : 1.0f;
  a.pos = pos;
  a.M = M;
  a.nh = nh;
  a.nkv = nkv;
  a.eps = eps;
  a.gq = gq;
  a.gk = gk;
  a.parts = rope_parts(M, nh + nkv, hd);
  return a;
}

}  // namespace
}  // namespace ws

using namespace ws;

extern "C" {

ws_status ws_rope_turns(const double* inv_freq, int32_t n, uint64_t* turns) {
  if (!inv_freq || !turns) return WS_ERR_INVALID;
  if (n < 1) return WS_ERR_SHAPE;
  for (int32_t i = 0; i < n; ++i) {
    if (!isfinite(inv_freq[i])) return WS_ERR_INVALID;
    double t = inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
    t -= floor(t);
    const double scaled = ldexp(t, 64);
    turns[i] = scaled >= 18446744073709551616.0 ? 0 : (uint64_t)scaled;
  }
  return WS_OK;
}

ws_status ws_qk_norm_rope_fwd(const ws_rope* rope, const int32_t* positions, int64_t M, int32_t n_heads,
                              int32_t n_kv_heads, int32_t head_dim, float eps, const float* q_gain,
                              const float* k_gain, const uint16_t* q, int64_t q_stride, const uint16_t* k,
                              int64_t k_stride, uint16_t* q_out, int64_t q_out_stride, uint16_t* k_out,
                              int64_t k_out_stride, ws_stream_t stream) {
  ws_status s = rope_shape(M, n_heads, n_kv_heads, head_dim);
  if (s != WS_OK) return s;
  if ((s = check_rope(rope, positions, q_gain, k_gain, eps, head_dim)) != WS_OK) return s;
  if ((s = check_io(q, q_stride, n_heads, head_dim)) != WS_OK) return s;
  if ((s = check_io(k, k_stride, n_kv_heads, head_dim)) != WS_OK) return s;
  if ((s = check_io(q_out, q_out_stride, n_heads, head_dim)) != WS_OK) return s;
  if ((s = check_io(k_out, k_out_stride, n_kv_heads, head_dim)) != WS_OK) return s;
  if (!same_rows(q, q_stride, q_out, q_out_stride) || !same_rows(k, k_stride, k_out, k_out_stride))
    return WS_ERR_INVALID;
  RopeArgs a = rope_args(rope, positions, M, n_heads, n_kv_heads, head_dim, eps, q_gain, k_gain);
  a.q = q;
  a.k = k;
  a.oq = q_out;
  a.ok = k_out;
  a.sq = q_stride;
  a.sk = k_stride;
  a.soq = q_out_stride;
  a.sok = k_out_stride;
  const bool il = rope && rope->interleaved;
  void (*kern)(const RopeArgs) = head_dim == 64 ? (il ? k_rope_fwd<64, true> : k_rope_fwd<64, false>)
                                                : (il ? k_rope_fwd<128, true> : k_rope_fwd<128, false>);
  note_launch();
  const cudaError_t e = launch_pdl(kern, dim3((unsigned)rope_ctas(M, a.parts, head_dim)), dim3(kRopeThreads),
                                   0, (cudaStream_t)stream, a);
  return e == cudaSuccess ? WS_OK : WS_ERR_CUDA;
}

ws_status ws_qk_norm_rope_workspace_size(int64_t M, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                         size_t* bytes) {
  if (!bytes) return WS_ERR_INVALID;
  const ws_status s = rope_shape(M, n_heads, n_kv_heads, head_dim);
  if (s != WS_OK) return s;
  const int parts = rope_parts(M, n_heads + n_kv_heads, head_dim, kGainThreads);
  *bytes = (size_t)rope_gain_ctas(M, parts, head_dim) * 2 * head_dim * 4;
  return WS_OK;
}

ws_status ws_qk_norm_rope_bwd(const ws_rope* rope, const int32_t* positions, int64_t M, int32_t n_heads,
                              int32_t n_kv_heads, int32_t head_dim, float eps, const float* q_gain,
                              const float* k_gain, const uint16_t* q, int64_t q_stride, const uint16_t* k,
                              int64_t k_stride, const uint16_t* dq_out, int64_t dq_out_stride,
                              const uint16_t* dk_out, int64_t dk_out_stride, uint16_t* dq,
                              int64_t dq_stride, uint16_t* dk, int64_t dk_stride, float* dq_gain,
                              float* dk_gain, int32_t accumulate, void* workspace, size_t ws_bytes,
                              ws_stream_t stream) {
  ws_status s = rope_shape(M, n_heads, n_kv_heads, head_dim);
  if (s != WS_OK) return s;
  if ((s = check_rope(rope, positions, q_gain, k_gain, eps, head_dim)) != WS_OK) return s;
  // without a norm the inputs are not read
  if (q_gain && (s = check_io(q, q_stride, n_heads, head_dim)) != WS_OK) return s;
  if (k_gain && (s = check_io(k, k_stride, n_kv_heads, head_dim)) != WS_OK) return s;
  if ((s = check_io(dq_out, dq_out_stride, n_heads, head_dim)) != WS_OK) return s;
  if ((s = check_io(dk_out, dk_out_stride, n_kv_heads, head_dim)) != WS_OK) return s;
  if ((s = check_io(dq, dq_stride, n_heads, head_dim)) != WS_OK) return s;
  if ((s = check_io(dk, dk_stride, n_kv_heads, head_dim)) != WS_OK) return s;
  if (!same_rows(dq_out, dq_out_stride, dq, dq_stride) || !same_rows(dk_out, dk_out_stride, dk, dk_stride) ||
      (q_gain && !same_rows(q, q_stride, dq, dq_stride)) || (k_gain && !same_rows(k, k_stride, dk, dk_stride)))
    return WS_ERR_INVALID;
  if (accumulate & ~WS_ACC_GRADS) return WS_ERR_INVALID;
  if ((dq_gain && !q_gain) || (dk_gain && !k_gain)) return WS_ERR_INVALID;
  if ((dq_gain && !al4r(dq_gain)) || (dk_gain && !al4r(dk_gain))) return WS_ERR_ALIGN;
  const bool gains = dq_gain || dk_gain;
  RopeArgs a = rope_args(rope, positions, M, n_heads, n_kv_heads, head_dim, eps, q_gain, k_gain);
  if (gains) a.parts = rope_parts(M, n_heads + n_kv_heads, head_dim, kGainThreads);
  const int64_t ctas = gains ? rope_gain_ctas(M, a.parts, head_dim) : rope_ctas(M, a.parts, head_dim);
  if (gains) {
    if (!workspace) return WS_ERR_INVALID;
    if (!al16r(workspace)) return WS_ERR_ALIGN;
    if (ws_bytes < (size_t)ctas * 2 * head_dim * 4) return WS_ERR_OOM;
  }
  a.q = q;
  a.k = k;
  a.uq = dq_out;
  a.uk = dk_out;
  a.oq = dq;
  a.ok = dk;
  a.sq = q_stride;
  a.sk = k_stride;
  a.suq = dq_out_stride;
  a.suk = dk_out_stride;
  a.soq = dq_stride;
  a.sok = dk_stride;
  a.partial = static_cast<float*>(workspace);
  const bool il = rope && rope->interleaved;
  void (*kern)(const RopeArgs);
  if (head_dim == 64)
    kern = gains ? (il ? k_rope_bwd<64, true, true> : k_rope_bwd<64, false, true>)
                 : (il ? k_rope_bwd<64, true, false> : k_rope_bwd<64, false, false>);
  else
    kern = gains ? (il ? k_rope_bwd<128, true, true> : k_rope_bwd<128, false, true>)
                 : (il ? k_rope_bwd<128, true, false> : k_rope_bwd<128, false, false>);
  note_launch();
  cudaError_t e = launch_pdl(kern, dim3((unsigned)ctas), dim3(kRopeThreads), 0, (cudaStream_t)stream, a);
  if (e == cudaSuccess && gains) {
    note_launch();
    e = launch_pdl(k_rope_gain, dim3((unsigned)(2 * head_dim / 32)), dim3(32 * kGainRows), 0,
                   (cudaStream_t)stream, (const float*)a.partial, (int)ctas, (int)head_dim, dq_gain, dk_gain,
                   (int)(accumulate & WS_ACC_GRADS));
  }
  return e == cudaSuccess ? WS_OK : WS_ERR_CUDA;
}

}  // extern "C"
