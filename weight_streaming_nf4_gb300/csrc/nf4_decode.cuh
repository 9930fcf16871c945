// nf4_decode.cuh -- NF4 codes to bf16 values in registers, the asynchronous
// global -> shared copies of the kernels that stage codes or activations, and
// the warp-wide matrix product of the many-adapter kernels.
#pragma once
#include "common.cuh"

namespace ws {

// Two IEEE fp32 products (round to nearest) in one packed instruction.
WS_DEVINL void mul2_rn(float x0, float x1, float s, float& r0, float& r1) {
  asm("{\n .reg .b64 pa, pb, pd;\n mov.b64 pa, {%2, %3};\n mov.b64 pb, {%4, %4};\n"
      " mul.rn.f32x2 pd, pa, pb;\n mov.b64 {%0, %1}, pd;\n}"
      : "=f"(r0), "=f"(r1)
      : "f"(x0), "f"(x1), "f"(s));
}

// Byte permute: bytes of {b, a} (a = bytes 0-3, b = 4-7) picked by the four
// 4-bit fields of sel.
WS_DEVINL uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// The 16 dequantised values of one 64-weight block, T[i] = bf16_RN(c_i * a)
// (one fp32 product, one rounding), split into byte planes: lo[q] holds the
// low bytes of T[4q..4q+3], hi[q] their high bytes.  A 4-bit code then
// becomes a bf16 value with byte permutes in registers -- no shared-memory
// table lookup per weight.
struct Nf4Table {
  uint32_t lo[4], hi[4];
};
WS_DEVINL Nf4Table make_table(float a) {
  uint32_t R[8];
  float v0, v1;
  mul2_rn(-1.0f, -0.6962f, a, v0, v1);
  R[0] = pack_bf16x2(v0, v1);
  mul2_rn(-0.5251f, -0.3949f, a, v0, v1);
  R[1] = pack_bf16x2(v0, v1);
  mul2_rn(-0.2844f, -0.1848f, a, v0, v1);
  R[2] = pack_bf16x2(v0, v1);
  mul2_rn(-0.0911f, 0.0f, a, v0, v1);
  R[3] = pack_bf16x2(v0, v1);
  mul2_rn(0.0796f, 0.1609f, a, v0, v1);
  R[4] = pack_bf16x2(v0, v1);
  mul2_rn(0.2461f, 0.3379f, a, v0, v1);
  R[5] = pack_bf16x2(v0, v1);
  mul2_rn(0.4407f, 0.5626f, a, v0, v1);
  R[6] = pack_bf16x2(v0, v1);
  mul2_rn(0.7230f, 1.0f, a, v0, v1);
  R[7] = pack_bf16x2(v0, v1);
  Nf4Table t;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    t.lo[q] = prmt(R[2 * q], R[2 * q + 1], 0x6420u);
    t.hi[q] = prmt(R[2 * q], R[2 * q + 1], 0x7531u);
  }
  return t;
}

// 4 code bytes (8 consecutive weights along k: byte i holds k = 2i in its
// high nibble, 2i+1 in its low nibble) -> 8 bf16 values in k order.
// Nibble f of the word is the code of k = f ^ 1; the two interleaving
// permutes at the end put the pairs back in k order, so the codes need no
// nibble swap first.
WS_DEVINL uint4 dq8(uint32_t w, const Nf4Table& t) {
  const uint32_t s7 = w & 0x77777777u;                           // index within 8 entries
  const uint32_t s8 = ((w >> 1) & 0x44444444u) | 0x32103210u;    // which half (code >= 8)
  uint32_t o[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a7 = h ? (s7 >> 16) : s7;
    const uint32_t a8 = h ? (s8 >> 16) : s8;
    // byte p of lo / hi: low / high byte of the value of nibble 4h + p
    const uint32_t lo = prmt(prmt(t.lo[0], t.lo[1], a7), prmt(t.lo[2], t.lo[3], a7), a8);
    const uint32_t hi = prmt(prmt(t.hi[0], t.hi[1], a7), prmt(t.hi[2], t.hi[3], a7), a8);
    o[2 * h] = prmt(lo, hi, 0x4051u);      // k = 4h (nibble 4h+1), k = 4h+1 (nibble 4h)
    o[2 * h + 1] = prmt(lo, hi, 0x6273u);  // k = 4h+2 (nibble 4h+3), k = 4h+3 (nibble 4h+2)
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Asynchronous 16- / 8- / 4-byte global -> shared copies; src_bytes = 0
// fills zeros without reading.
WS_DEVINL void cp_async16(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(src_bytes)
               : "memory");
}
WS_DEVINL void cp_async8(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(src_bytes)
               : "memory");
}
WS_DEVINL void cp_async4(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes)
               : "memory");
}
WS_DEVINL void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
WS_DEVINL void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), bf16.  Lane (g = lane / 4, t =
// lane % 4) holds A rows g, g + 8 at k = 2t, 2t+1 (a0, a1) and 2t+8, 2t+9 (a2,
// a3); B column g at the same k (b0, b1); D rows g (d[0], d[1]) and g + 8 at
// columns 2t, 2t+1.  The kernels that use it permute the contraction index
// (alike in A and B), so that a lane's elements are contiguous in memory.
WS_DEVINL void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace ws
