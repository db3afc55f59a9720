// nt_kv8.cuh -- layout and checks of the paged 8-bit K/V cache (include/nt.h,
// nt_kv8_cache), shared by its operators (nt_kv8.cu), the selection of pages
// (nt_kv8_select.cu) and the attention over it (nt_kv8_attn.cu).  Tables, lengths,
// counts, row lists and page operators are those of the 4-bit cache (nt_kv4.cuh).
#pragma once

#include "nt_kv4.cuh"

namespace nt {

constexpr int kKv8MaxGroup = 16;                   // query heads per kv head
constexpr int kKv8MinExp = -100;
constexpr float kKv8Most = 448.f * 0x1p100f;       // largest magnitude that can be held

// Offsets inside a page.  Per kv head: K codes, V codes; behind all of them per kv head
// the exponents (16 bytes, two used) and the bounds lo [hd], hi [hd].
struct Kv8Page {
  int hd, page_len, n_kv;
  __host__ __device__ explicit Kv8Page(const Kv4& c) : hd(c.hd), page_len(c.page_len), n_kv(c.n_kv) {}
  __host__ __device__ int codes() const { return page_len * hd; }
  __host__ __device__ int64_t k(int g) const { return int64_t(g) * 2 * codes(); }
  __host__ __device__ int64_t v(int g) const { return k(g) + codes(); }
  __host__ __device__ int64_t exps(int g) const { return int64_t(n_kv) * 2 * codes() + int64_t(g) * (16 + 2 * hd); }
  __host__ __device__ int64_t bounds(int g) const { return exps(g) + 16; }
  __host__ __device__ int64_t bytes() const { return exps(n_kv); }
};
// 16 codes of position t from dimension 16 ch on; of dimension d from position 16 tc on
__host__ __device__ __forceinline__ int kv8_k_at(int hd, int t, int ch) { return (t >> 3) * 8 * hd + ch * 128 + (t & 7) * 16; }
__host__ __device__ __forceinline__ int kv8_v_at(int hd, int tc, int d) { return (tc * hd + d) * 16; }

nt_status kv8_check(const nt_kv8_cache* c, const char* who, bool pointers, Kv4* k);

// Bytes of the workspace of the selection and of the attention.
size_t kv8_select_ws_bytes(const Kv4& k, int64_t n);
size_t kv8_attn_ws_bytes(int hd);

// ------------------------------------------------------------ device helpers --

__device__ __forceinline__ float kv8_exp2i(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }   // |e| <= 126

// Exponent of a page whose largest magnitude is `top` (finite, at most kKv8Most): 448 is 1.75 2^8.
__device__ __forceinline__ int kv8_exponent(float top) {
  const uint32_t b = __float_as_uint(top);
  const int e = int(b >> 23) - 135 + ((b & 0x7fffffu) > 0x600000u);
  return e < kKv8MinExp ? kKv8MinExp : e;
}
__device__ __forceinline__ bool kv8_held(float x) { return fabsf(x) <= kKv8Most; }   // (not NaN)

// Sequence of entry i (seq0 + i where none are listed) and the positions that it sees (-1 and none: cannot be read, the bit in *bad).
__device__ __forceinline__ int2 kv8_entry(const Kv4& c, const int32_t* seq, const int32_t* ctx, int seq0, int i, uint32_t* bad) {
  const int s = seq ? seq[i] : seq0 + i;
  *bad = NT_KV4_BAD_SEQ;
  if (s < 0 || s >= c.max_seqs) return make_int2(-1, 0);
  const int len = c.len[s], n = ctx ? ctx[i] : len;
  *bad = len < 0 || len > c.capacity() || n < 0 || n > len ? NT_KV4_BAD_LEN : 0;
  return make_int2(*bad ? -1 : s, *bad ? 0 : n);
}

// Codes of two values, the first in the low byte.
__device__ __forceinline__ uint32_t kv8_code2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// what is coded of a value in a page of exponent e (up = 2^-e)
__device__ __forceinline__ float kv8_scaled(float x, float up) { return kv8_held(x) ? x * up : NAN; }
__device__ __forceinline__ float2 kv8_value2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(codes)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint32_t kv8_code4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// the values of four codes as f16 pairs
__device__ __forceinline__ void kv8_half4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// two fp32 numbers at a time
__device__ __forceinline__ uint64_t kv8_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 kv8_unpack(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ uint64_t kv8_mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t kv8_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Four codes rounded again for an exponent larger by the one that f = 2^-it stands for.
__device__ __forceinline__ uint32_t kv8_again(uint32_t w, float f) {
  const float2 a = kv8_value2(w & 0xffffu), b = kv8_value2(w >> 16);
  return kv8_code4(a.x * f, a.y * f, b.x * f, b.y * f);
}
__device__ __forceinline__ uint4 kv8_again(uint4 w, float f) {
  return make_uint4(kv8_again(w.x, f), kv8_again(w.y, f), kv8_again(w.z, f), kv8_again(w.w, f));
}

}  // namespace nt
