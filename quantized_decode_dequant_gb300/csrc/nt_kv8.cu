// nt_kv8.cu -- the paged 8-bit K/V cache: rows into it, with the position rotation, and
// out of it, and its page operators (include/nt.h documents each).
#include "nt_kv8.cuh"

#include <cmath>

namespace nt {

nt_status kv8_check(const nt_kv8_cache* c, const char* who, bool pointers, Kv4* k) {
  if (!c) return fail(NT_E_INVAL, std::string(who) + ": NULL cache");
  if (c->page_len != 16 && c->page_len != 32 && c->page_len != 64 && c->page_len != 128)
    return fail(c->page_len < 1 ? NT_E_INVAL : NT_E_UNSUPPORTED, std::string(who) + ": page_len must be 16, 32, 64 or 128");
  *k = Kv4{c->n_layers, c->n_kv_heads, c->head_dim, c->page_len, c->n_pages, c->max_seqs, c->max_pages,
           static_cast<uint8_t*>(c->pool), c->table, c->len, c->refs, c->error, 0};
  k->pb = Kv8Page(*k).bytes();
  return kv4_check_pages(*k, who, pointers);
}

// ------------------------------------------------------------ the rotation --
//
// cos and sin of position p's angle p f to about 2^-45: the angle in turns is a 64-bit
// fraction, p times the frequency's, so that reducing it costs nothing and no position is
// too far; its first 8 bits (rounded) pick a point of the circle, held as two fp32 terms each; what
// is left, at most pi / 256, goes through the first terms of the series, and the two are
// multiplied in pairs of fp32.  (In fp64 it would take the few units that this GPU has
// for it; in plain fp32 a key next to the border of two codes would get the wrong one
// about once in 10^6 values.)

struct __align__(16) Kv8Point {
  float c, cl, s, sl;   // cos, sin: the sums of two terms
};
struct Kv8Circle {
  Kv8Point p[256];
};
constexpr double kv8_series(double x, bool sine) {   // |x| <= pi / 4
  double term = sine ? x : 1.0, sum = term;
  for (int i = sine ? 2 : 1; i < 30; i += 2) {
    term *= -x * x / (double(i) * (i + 1));
    sum += term;
  }
  return sum;
}
constexpr Kv8Circle kv8_circle() {
  constexpr double kPi = 3.14159265358979323846;
  Kv8Circle t{};
  for (int i = 0; i < 256; i++) {
    const int quarter = (i + 32) / 64, off = i - 64 * quarter;         // off in [-32, 32)
    const double x = off * kPi / 128, cc = kv8_series(x, false), ss = kv8_series(x, true);
    const double c = quarter % 4 == 0 ? cc : quarter % 4 == 1 ? -ss : quarter % 4 == 2 ? -cc : ss;
    const double s = quarter % 4 == 0 ? ss : quarter % 4 == 1 ? cc : quarter % 4 == 2 ? -ss : -cc;
    t.p[i].c = float(c);
    t.p[i].cl = float(c - double(t.p[i].c));
    t.p[i].s = float(s);
    t.p[i].sl = float(s - double(t.p[i].s));
  }
  return t;
}
__device__ constexpr Kv8Circle kKv8Circle = kv8_circle();   // (kernels look points up in a copy in shared memory, `circle`)

// a + b in two terms (a in hi already: hi = a + b rounded)
__device__ __forceinline__ float kv8_rest(float a, float b, float hi) {
  const float bb = __fsub_rn(hi, a);
  return __fadd_rn(__fsub_rn(a, __fsub_rn(hi, bb)), __fsub_rn(b, bb));
}
__device__ __forceinline__ Kv8Point kv8_turn(const Kv8Point* circle, uint64_t phase, int pos) {
  const uint64_t turn = phase * uint64_t(uint32_t(pos));
  const uint32_t i = uint32_t((turn + (1ull << 55)) >> 56) & 255u;
  const int64_t rest = int64_t(turn - (uint64_t(i) << 56));                  // in [-2^55, 2^55)
  const float a = float(int32_t(rest >> 32)), b = float(uint32_t(rest) >> 8);   // exact
  // r = 2 pi (a 2^-32 + b 2^-56)
  constexpr double k = 6.283185307179586477 * 0x1p-32;
  constexpr float kh = float(k), kl = float(k - double(kh)), kb = float(k * 0x1p-24);
  const float r = __fmul_rn(a, kh), rl = __fadd_rn(__fmaf_rn(a, kh, -r), __fmaf_rn(a, kl, __fmul_rn(b, kb)));
  const float q = __fmul_rn(r, r), ql = __fmaf_rn(2.f * r, rl, __fmaf_rn(r, r, -q));
  // sin r and cos r - 1
  const float s = r, sl = __fsub_rn(rl, __fmul_rn(__fmul_rn(q, r), __fmaf_rn(q, -1.f / 120.f, 1.f / 6.f)));
  const float m = -0.5f * q, ml = __fmaf_rn(__fmul_rn(q, q), __fmaf_rn(q, -1.f / 720.f, 1.f / 24.f), -0.5f * ql);
  const float4 at = *reinterpret_cast<const float4*>(&circle[i]);
  const float C = at.x, Cl = at.y, S = at.z, Sl = at.w;
  auto times = [](float x, float xl, float y, float yl, float& p) {          // (x + xl) (y + yl) = p + the rest
    p = __fmul_rn(x, y);
    return __fadd_rn(__fmaf_rn(x, y, -p), __fmaf_rn(x, yl, __fmul_rn(xl, y)));
  };
  Kv8Point t;
  float p1, p2;
  const float e1 = times(C, Cl, m, ml, p1), e2 = times(S, Sl, s, sl, p2);
  const float d = __fsub_rn(p1, p2);
  t.c = __fadd_rn(C, d);
  t.cl = __fadd_rn(kv8_rest(C, d, t.c), __fadd_rn(kv8_rest(p1, -p2, d), __fadd_rn(__fsub_rn(e1, e2), Cl)));
  const float e3 = times(S, Sl, m, ml, p1), e4 = times(C, Cl, s, sl, p2);
  const float u = __fadd_rn(p1, p2);
  t.s = __fadd_rn(S, u);
  t.sl = __fadd_rn(kv8_rest(S, u, t.s), __fadd_rn(kv8_rest(p1, p2, u), __fadd_rn(__fadd_rn(e3, e4), Sl)));
  return t;
}
// a c + b s, rounded once but for about 2^-45 of the products
__device__ __forceinline__ float kv8_dot2(float a, float c, float cl, float b, float s, float sl) {
  const float p = __fmul_rn(a, c), q = __fmul_rn(b, s), d = __fadd_rn(p, q);
  const float e = __fmaf_rn(a, cl, __fmaf_rn(a, c, -p)), f = __fmaf_rn(b, sl, __fmaf_rn(b, s, -q));
  const float r = __fadd_rn(d, __fadd_rn(kv8_rest(p, q, d), __fadd_rn(e, f)));
  return fabsf(r) <= 3.4028234e38f && (r != 0.f || d != 0.f) ? r : d;   // (an infinity leaves no rest, a zero keeps its sign)
}
__device__ __forceinline__ void kv8_rotate(const Kv8Point& t, float& a, float& b) {
  const float x = kv8_dot2(a, t.c, t.cl, b, -t.s, -t.sl);
  b = kv8_dot2(a, t.s, t.sl, b, t.c, t.cl);
  a = x;
}

// cos and sin in fp32, off by less than 2^-24.8 (of 1).  In units of 2^-25: the last addition rounds (1); the angle r, at most
// pi / 256, loses the turn's lower half, 2 pi 2^-32 (0.05); rounding r, its factor and sin r, and the two inner sums of at most 2^-6 each,
// 2^-31 (0.08 in all); cos r - 1, the series' next terms and the points' second terms are below 2^-36.  1.13, 2^-24.82.
__device__ __forceinline__ float2 kv8_turn_fast(const Kv8Point* circle, uint64_t turn) {
  const uint32_t i = uint32_t((turn + (1ull << 55)) >> 56) & 255u;
  constexpr float k = float(6.283185307179586477 * 0x1p-32);
  const float r = float(int32_t(uint32_t(turn >> 32) - (i << 24))) * k, q = r * r;
  const float s = fmaf(r * q, -1.f / 6.f, r), m = q * fmaf(q, 1.f / 24.f, -0.5f);
  const float4 at = *reinterpret_cast<const float4*>(&circle[i]);
  return make_float2(at.x + fmaf(at.x, m, fmaf(-at.z, s, at.y)), at.z + fmaf(at.z, m, fmaf(at.x, s, at.w)));
}

// ------------------------------------------------------------ append, read --
//
// append: a CTA takes the K or the V of one page of one sequence, the rows that fall on its positions, for several kv heads
// one after the other, the next one's rows on the way; the page's exponent needs all rows of a head before the first code.  A
// thread has 32 values: of K 4 dimensions of 8 positions (cos and sin of the page's positions stand in shared memory for
// all heads, and four threads exchange their codes for runs of 16), of V 2 dimensions of 16 positions (a run each).
//   A key is rotated in fp32, which is off by less than d = 1.25 2^-22 (|x| + |y|) of its pair (kUnsure).  Where x + d and
// x - d have different codes (about one value in 10^4), the warp puts the key on a list and forms it again to 2^-45 when all
// heads are through, one key a lane, in place of 1000 cycles and more that the other warps would wait for at the next head's
// barrier; where the largest magnitude of a warp lies that near to where the exponent changes, the list is full or there is one
// head only, it does so at once.
//   What bounds it: 2 x 20011 f16 rows, 8 heads of 128, pages of 64 (247 MB in and out): 81 us, 3.0 TB/s.  A page's K takes a
// CTA 37,000 cycles, 8000 of them before the first head (its rows and page looked up, cos and sin), V 24,500; while V pages
// are stored, memory is the bound (6 TB/s of reads and writes), while K pages are, instructions and a barrier a head; and 626
// pages are little more than two rounds of 304 CTAs.  (More rows on the way, four heads by cp.async: 85 where it was 83.5;
// 3 CTAs an SM, 80 registers, spills: no gain; 16 positions of a head in a warp, the first form: 199.)  1 token: 4.5 us, a
// launch and five dependent reads.
// read: a warp handles K or V of 16 positions of one sequence and kv head; 2 x 20011 f16 rows: 40.6 us, 6.0 TB/s.

struct Kv8Rot {
  uint64_t phase[64];   // turns per position, as 64-bit fractions
  int32_t on, heads;
  int32_t q_heads;      // that a warp rotates, a multiple of 4
  int32_t splits, per;  // CTAs that share a page's kv heads, and heads (times those side by side) that each takes
  int64_t q_stride, out_stride;
  float* out;
};

// Heads of a page go one after the other in a CTA (cos and sin are formed once, the next rows are on the way), but not in fewer
// CTAs than this (of 256 threads; by the units of the call, of which entries of few rows use half).  (us with 1, 2, 4 and 8 heads of
// 128 a CTA: 500 rows 7.7, 9.5, 13.4, 20; 2000 rows 13.2, 10.7, 13.3, 21; 8000 rows 37, 28.5, 27.0, 27.9; 2 x 20011 rows
// 173, 122, 98, 88; 64 sequences of 1 row 22, 16.6, 14.2, 19.8.)
constexpr int kKv8AppendCtas = 3 * 152;
// Query heads that a warp rotates at its row's position (whose cos and sin cost as much as 4 heads): 16 or 8 where that leaves as many warps as
// this, else 4.  (us with 4, 8 and 16, heads of 128 in fp32: 100 rows of 32 heads 6.5, 6.1, 6.2; 500 of 64 12.5, 11.5, 11.9; 2000 of
// 32 30, 27.7, 26.5; 9000 of 64 213, 180, 159.)
constexpr int kKv8QWarps16 = 152 * 16, kKv8QWarps8 = 152;

template <class T> struct Kv8Quad;   // four elements of a source
template <> struct Kv8Quad<float> {
  static __device__ __forceinline__ float4 get(const float* p) { return *reinterpret_cast<const float4*>(p); }
};
template <> struct Kv8Quad<__half> {
  static __device__ __forceinline__ float4 get(const __half* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
    return make_float4(a.x, a.y, b.x, b.y);
  }
};

// Position of row `row` of the call, below 0 where it belongs to no entry that can be read.
__device__ __forceinline__ int kv8_row_pos(const Kv4& c, const Kv4Rows& a, int row) {
  int i = row, b0 = row, b1 = row + 1;
  if (a.begin) {
    int lo = 0, hi = a.n;   // the last entry that begins at or before the row
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.begin[mid] <= row) lo = mid; else hi = mid;
    }
    i = lo;
    b0 = a.begin[i];
    b1 = a.begin[i + 1];
    if (b0 < 0 || row < b0 || row >= b1 || b1 > a.n_rows) return -1;
  } else if (row >= a.n) {
    return -1;
  }
  const int s = a.seq ? a.seq[i] : i;
  if (s < 0 || s >= c.max_seqs) return -1;
  const int n = c.len[s];
  if (n > c.capacity() || n < b1 - b0) return -1;
  return n - (b1 - row);
}

template <int HD, class T>
__device__ __forceinline__ void kv8_rotate_q(const Kv4& c, const Kv4Rows& a, const Kv8Rot& r, const Kv8Point* circle, const uint64_t* phase,
                                             const T* q, int64_t id) {
  constexpr int kLanes = HD / 4, kSide = 32 / kLanes, kFew = 4 / kSide;   // lanes of a head, heads side by side, on the way together
  const int lane = threadIdx.x & 31, groups = (r.heads + r.q_heads - 1) / r.q_heads;
  const int64_t unit = id * (blockDim.x / 32) + (threadIdx.x >> 5);
  if (unit >= int64_t(a.n_rows) * groups) return;
  const int row = int(unit / groups), h0 = int(unit % groups) * r.q_heads, h1 = min(h0 + r.q_heads, r.heads);
  const int pos = kv8_row_pos(c, a, row);
  if (pos < 0) return;
  const int i = lane % kLanes;
  const Kv8Point t0 = kv8_turn(circle, phase[2 * i], pos), t1 = kv8_turn(circle, phase[2 * i + 1], pos);
  const T* from = q + int64_t(row) * r.q_stride + 4 * i;
  float* to = r.out + int64_t(row) * r.out_stride + 4 * i;
#pragma unroll 1
  for (int h = h0 + lane / kLanes; h < h1; h += 4) {
    float4 x[kFew];
#pragma unroll
    for (int y = 0; y < kFew; y++)
      if (h + y * kSide < h1) x[y] = Kv8Quad<T>::get(from + (h + y * kSide) * HD);
#pragma unroll
    for (int y = 0; y < kFew; y++) {
      if (h + y * kSide >= h1) break;
      kv8_rotate(t0, x[y].x, x[y].y);
      kv8_rotate(t1, x[y].z, x[y].w);
      *reinterpret_cast<float4*>(to + (h + y * kSide) * HD) = x[y];
    }
  }
}

// Error of a rotated key in fp32, relative to S = |x| + |y| of its pair, in units of 2^-24: cos and sin are off by 2^-24.8, which (|a| +
// |b|) <= sqrt(2) S multiplies (0.82); the first product rounds (|b| <= S: 1), the multiply-add (1), and the key that the format defines is rounded to
// fp32 once itself (1); forming x 2^-e -+ d rounds (1).  4.82 2^-24 in all, where kUnsure is 5.
constexpr float kUnsure = 0x1.4p-22f;

// What the threads of an append know of their page.
struct Kv8Mine {
  uint8_t* base;         // the page
  int64_t row_stride;    // of the source
  int p0, pos0;          // first position within the page, and of the sequence
  int d0;                // first dimension
  int first, last;       // the page's new positions
  uint32_t live;         // bit i: position p0 + i is one of them
  bool fresh;
  __device__ __forceinline__ bool has(int i) const { return live >> i & 1u; }
};
template <int HD, int NT>
struct Kv8AppendShared {
  static constexpr int kGroups = NT / (HD / 4);     // of 8 positions, over all heads side by side
  uint64_t phase[HD / 2];
  int exp[2][NT / 32];
  uint32_t lo[2][kGroups * HD / 2], hi[2][kGroups * HD / 2];   // f16 pairs
  Kv8Point circle[256];
  uint32_t later[NT / 32][32];                      // a warp's keys to be formed again: step, lane, position of eight
};
extern __shared__ __align__(16) float kv8_turns[];   // [position of the page][pair / 2]: cos of both pairs, sin of both

// Keys of the positions in `which` (of 8; 4 dimensions each) to 2^-45, into out [8][4].
template <class T>
__device__ __noinline__ void kv8_exact_keys(const T* from, int64_t row_stride, uint32_t which, bool turned, const Kv8Point* circle,
                                            const uint64_t* phase, int pos0,
                                            float* out) {
#pragma unroll 1
  for (int i = 0; i < 8; i++) {
    if (!(which >> i & 1u)) continue;
    float4 y = Kv8Quad<T>::get(from + i * row_stride);
    if (turned) {
      kv8_rotate(kv8_turn(circle, phase[0], pos0 + i), y.x, y.y);
      kv8_rotate(kv8_turn(circle, phase[1], pos0 + i), y.z, y.w);
    }
    out[4 * i] = kv8_held(y.x) ? y.x : NAN;
    out[4 * i + 1] = kv8_held(y.y) ? y.y : NAN;
    out[4 * i + 2] = kv8_held(y.z) ? y.z : NAN;
    out[4 * i + 3] = kv8_held(y.w) ? y.w : NAN;
  }
}

// The key quad at `from` to 2^-45, as codes.
template <class T>
__device__ __forceinline__ uint32_t kv8_exact_codes(const T* from, bool turned, const Kv8Point* circle, const uint64_t* phase, int pos,
                                                    float up) {
  float4 y = Kv8Quad<T>::get(from);
  if (turned) {
    kv8_rotate(kv8_turn(circle, phase[0], pos), y.x, y.y);
    kv8_rotate(kv8_turn(circle, phase[1], pos), y.z, y.w);
  }
  return kv8_code4(kv8_scaled(y.x, up), kv8_scaled(y.y, up), kv8_scaled(y.z, up), kv8_scaled(y.w, up));
}

template <class T> struct Kv8Raw;   // what a thread has of a head as it comes: 8 times 4 (K) or 16 times 2 (V) elements
template <> struct Kv8Raw<float> {
  static constexpr int kWords = 32;
  static __device__ __forceinline__ void get4(const float* p, uint32_t* w) {
    const uint4 y = *reinterpret_cast<const uint4*>(p);
    w[0] = y.x; w[1] = y.y; w[2] = y.z; w[3] = y.w;
  }
  static __device__ __forceinline__ void get2(const float* p, uint32_t* w) {
    const uint2 y = *reinterpret_cast<const uint2*>(p);
    w[0] = y.x; w[1] = y.y;
  }
  static __device__ __forceinline__ float2 pair(const uint32_t* w, int i) { return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])); }
};
template <> struct Kv8Raw<__half> {
  static constexpr int kWords = 16;
  static __device__ __forceinline__ void get4(const __half* p, uint32_t* w) {
    const uint2 y = *reinterpret_cast<const uint2*>(p);
    w[0] = y.x; w[1] = y.y;
  }
  static __device__ __forceinline__ void get2(const __half* p, uint32_t* w) { w[0] = *reinterpret_cast<const uint32_t*>(p); }
  static __device__ __forceinline__ float2 pair(const uint32_t* w, int i) { return __half22float2(*reinterpret_cast<const __half2*>(w + i)); }
};

__device__ __forceinline__ uint32_t kv8_min2(uint32_t a, uint32_t b) {   // of f16 pairs, NaN where one is
  uint32_t d;
  asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t kv8_max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

template <class T, bool V>
__device__ __forceinline__ void kv8_load(const Kv8Mine& me, const T* from, bool on, uint32_t (&w)[Kv8Raw<T>::kWords]) {
  constexpr int N = V ? 16 : 8, E = Kv8Raw<T>::kWords / N;
#pragma unroll
  for (int i = 0; i < N; i++) {
    if (on && me.has(i)) {
      if (V) Kv8Raw<T>::get2(from, w + E * i); else Kv8Raw<T>::get4(from, w + E * i);
    } else {
#pragma unroll
      for (int j = 0; j < E; j++) w[E * i + j] = 0u;
    }
    from += me.row_stride;
  }
}

// Largest magnitude of a warp's values, NaN passed over (infinities and what lies beyond the largest that can be held are the caller's affair).
__device__ __forceinline__ float kv8_largest(const float (&x)[32]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 32; i += 2) m = fmaxf(m, fmaxf(fabsf(x[i]), fabsf(x[i + 1])));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}

// Codes of a head's V: a thread's 2 dimensions of 16 positions, a run each.
template <int HD>
__device__ __forceinline__ void kv8_put_v(const Kv8Mine& me, const float (&x)[32], uint8_t* to, float up, bool again, float f) {
  uint32_t w[2][4];
#pragma unroll
  for (int j = 0; j < 2; j++)
#pragma unroll
    for (int i = 0; i < 4; i++) w[j][i] = kv8_code4(x[8 * i + j] * up, x[8 * i + 2 + j] * up, x[8 * i + 4 + j] * up, x[8 * i + 6 + j] * up);
  uint4* at = reinterpret_cast<uint4*>(to + kv8_v_at(HD, me.p0 >> 4, me.d0));
  if (me.live == 0xffffu) {
#pragma unroll
    for (int j = 0; j < 2; j++) at[j] = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
    return;
  }
  // positions of this run: new [first, last), older below
  const int first = max(me.first - me.p0, 0), last = min(me.last - me.p0, 16);
  if (!(last > first || (again && first > 0))) return;
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const uint4 was = at[j];
    const uint32_t old[4] = {was.x, was.y, was.z, was.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      auto below = [&](int n) { n -= 4 * i; return n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u; };   // bytes of positions below n
      const uint32_t older = below(first < 16 ? first : 16), mine = below(last) & ~older;
      const uint32_t kept = again ? kv8_again(old[i], f) : old[i];
      w[j][i] = (w[j][i] & mine) | (kept & older) | (old[i] & ~(mine | older));
    }
    at[j] = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
  }
}

// Codes of a head's K: a thread's 4 dimensions of 8 positions (w), which four threads exchange for 16 dimensions of 2 positions each.
template <int HD>
__device__ __forceinline__ void kv8_put_k(const Kv8Mine& me, uint32_t (&w)[8], uint8_t* to, bool on, bool again, float f) {
  const int n = threadIdx.x & 3;
  // w[2 m + b] is position 2 m + b: exchange the m of threads whose n differs in bit 1, then in bit 0
#pragma unroll
  for (int b = 0; b < 2; b++) {
#pragma unroll
    for (int m = 0; m < 2; m++) {
      const uint32_t give = n & 2 ? w[2 * m + b] : w[2 * (m + 2) + b], got = __shfl_xor_sync(0xffffffffu, give, 2);
      if (n & 2) w[2 * m + b] = got; else w[2 * (m + 2) + b] = got;
    }
#pragma unroll
    for (int m = 0; m < 4; m += 2) {
      const uint32_t give = n & 1 ? w[2 * m + b] : w[2 * (m + 1) + b], got = __shfl_xor_sync(0xffffffffu, give, 1);
      if (n & 1) w[2 * m + b] = got; else w[2 * (m + 1) + b] = got;
    }
  }
  if (!on) return;
#pragma unroll
  for (int b = 0; b < 2; b++) {
    const int p = me.p0 + 2 * n + b;
    uint4* at = reinterpret_cast<uint4*>(to + kv8_k_at(HD, p, me.d0 >> 4));
    if (me.has(2 * n + b)) *at = make_uint4(w[b], w[2 + b], w[4 + b], w[6 + b]);
    else if (again && p < me.first) *at = kv8_again(*at, f);
  }
}

// K (or V) of a page for the kv heads g, g + abreast, ... below g1 and of the split's `steps`.
template <int HD, class T, int NT, bool V>
__device__ __forceinline__ void kv8_append_page(const Kv4& c, const Kv8Page& L, const Kv8Mine& me, Kv8AppendShared<HD, NT>& sh, const T* src,
                                                int64_t head_stride, bool turned, int g, int abreast, int steps,
                                                uint32_t (&raw)[Kv8Raw<T>::kWords]) {
  const int t = threadIdx.x, lane = t & 31, P = c.page_len, tph = P * HD / 32, hp = t / tph, th = t % tph, wph = tph / 32;
  const bool busy = __any_sync(0xffffffffu, me.live != 0u);            // the warp has new positions
  // The page's bounds of a head, two dimensions a thread, are put together behind the next head's barrier: one barrier a head.
  const bool two = !V && th < HD / 2;
  const int g0 = g;
  int later = 0;                                                       // keys on the warp's list
  int8_t* bounds = nullptr;                                            // of the head before (nullptr: none)
  char2 lo_was = make_char2(0, 0), hi_was = lo_was;
  float f_was = 1.f;
  auto join_bounds = [&](int buf) {
    if (V || !bounds) return;
    const int groups = P / 8;
    uint32_t least = 0x7c007c00u, most = 0xfc00fc00u;
#pragma unroll 4
    for (int y = 0; y < groups; y++) {
      least = kv8_min2(least, sh.lo[buf][(hp * groups + y) * (HD / 2) + th]);
      most = kv8_max2(most, sh.hi[buf][(hp * groups + y) * (HD / 2) + th]);
    }
    auto bound = [&](int j, int lo0, int hi0, int8_t& l1, int8_t& h1) {
      const float l = __half2float(__ushort_as_half(uint16_t(least >> (16 * j)))), h = __half2float(__ushort_as_half(uint16_t(most >> (16 * j))));
      // (infinities where every row's key is on a list)
      int lo1 = l != l ? -127 : min(int(floorf(l * 0.25f)), 127), hi1 = l != l ? 127 : max(int(ceilf(h * 0.25f)), -127);
      if (!me.fresh) {
        if (lo0 != -127) lo0 = int(floorf(lo0 * f_was));
        if (hi0 != 127) hi0 = int(ceilf(hi0 * f_was));
        lo1 = min(lo1, lo0);
        hi1 = max(hi1, hi0);
      }
      l1 = int8_t(lo1);
      h1 = int8_t(hi1);
    };
    int8_t l0, l1, h0, h1;
    bound(0, lo_was.x, hi_was.x, l0, h0);
    bound(1, lo_was.y, hi_was.y, l1, h1);
    *reinterpret_cast<char2*>(bounds) = make_char2(l0, l1);
    *reinterpret_cast<char2*>(bounds + HD) = make_char2(h0, h1);
    bounds = nullptr;
  };
#pragma unroll 1
  for (int step = 0; step < steps; step++, g += abreast) {
    const int buf = step & 1;
    const bool on = g < c.n_kv;
    int8_t* exps = reinterpret_cast<int8_t*>(me.base + L.exps(on ? g : 0)) + V;
    const int was = me.fresh ? kKv8MinExp : *exps;
    float x[32];
#pragma unroll
    for (int i = 0; i < 16; i++) {
      const float2 y = Kv8Raw<T>::pair(raw, i);
      x[2 * i] = y.x; x[2 * i + 1] = y.y;
    }
    const T* from = src + int64_t(g) * head_stride;
    if (step + 1 < steps) kv8_load<T, V>(me, from + int64_t(abreast) * head_stride, g + abreast < c.n_kv, raw);   // the next head's, on the way
    if (!V && turned && busy) {
      const float4* turn = reinterpret_cast<const float4*>(kv8_turns) + me.p0 * (HD / 4) + me.d0 / 4;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float4 z = turn[i * (HD / 4)];
        const float u0 = x[4 * i], u1 = x[4 * i + 1], u2 = x[4 * i + 2], u3 = x[4 * i + 3];
        x[4 * i] = fmaf(u0, z.x, -u1 * z.z);
        x[4 * i + 2] = fmaf(u2, z.y, -u3 * z.w);
        const float2 y = kv8_unpack(kv8_fma2(kv8_pack(u0, u2), kv8_pack(z.z, z.w), kv8_mul2(kv8_pack(u1, u3), kv8_pack(z.x, z.y))));
        x[4 * i + 1] = y.x;
        x[4 * i + 3] = y.y;
      }
    }
    bool exact = V || !turned;
    float top = kv8_largest(x);
    constexpr uint32_t kNear = 64;                                     // of 2^-23: farther than the error of x (S is at most twice the largest)
    const uint32_t from_border = (__float_as_uint(top) & 0x7fffffu) - (0x600000u - kNear);
    if (__float_as_uint(top) > __float_as_uint(kKv8Most) - kNear || (!exact && from_border <= 2 * kNear)) {
      if (V) {
#pragma unroll
        for (int i = 0; i < 32; i++) x[i] = kv8_held(x[i]) ? x[i] : NAN;
      } else {
        float y[32];
#pragma unroll
        for (int i = 0; i < 32; i++) y[i] = 0.f;
        kv8_exact_keys(from, me.row_stride, on ? me.live : 0u, turned, sh.circle, sh.phase + me.d0 / 2, me.pos0, y);
#pragma unroll
        for (int i = 0; i < 32; i++) x[i] = y[i];
      }
      exact = true;
      top = kv8_largest(x);
    }
    if (lane == 0) sh.exp[buf][t >> 5] = kv8_exponent(top);
    __syncthreads();
    join_bounds(buf ^ 1);
    if (two && on) {
      bounds = reinterpret_cast<int8_t*>(me.base + L.bounds(g)) + 2 * th;
      if (!me.fresh) {
        lo_was = *reinterpret_cast<const char2*>(bounds);
        hi_was = *reinterpret_cast<const char2*>(bounds + HD);
      }
    }
    const int e = max(was, __reduce_max_sync(0xffffffffu, lane < wph ? sh.exp[buf][hp * wph + lane] : kKv8MinExp));
    const float up = kv8_exp2i(-e);
    const int less = e - was;                                          // exponents that older codes are rounded for
    const bool again = !me.fresh && less > 0;
    const float f = kv8_exp2i(less > 126 ? -126 : -less);              // (from 2^-20 on every code is rounded to zero)
    if (V) {
      if (on) kv8_put_v<HD>(me, x, me.base + L.v(g), up, again, f);
    } else {
      uint32_t lo[2] = {0x7c007c00u, 0x7c007c00u}, hi[2] = {0xfc00fc00u, 0xfc00fc00u};   // bounds of this thread's positions
      uint32_t w[8] = {}, mine = me.live;                              // mine: of whose keys the codes are right
      if (busy) {
        uint32_t z[8], differ = 0u;                                      // codes of a position's 4 dimensions, of x - d and x + d
        const uint64_t up2 = kv8_pack(up, up), off = kv8_pack(up * kUnsure, up * kUnsure), minus = kv8_pack(up * -kUnsure, up * -kUnsure);
        if (exact) {
#pragma unroll
          for (int i = 0; i < 8; i++) w[i] = z[i] = kv8_code4(x[4 * i] * up, x[4 * i + 1] * up, x[4 * i + 2] * up, x[4 * i + 3] * up);
        } else {
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const uint64_t x02 = kv8_pack(x[4 * i], x[4 * i + 2]), x13 = kv8_pack(x[4 * i + 1], x[4 * i + 3]);
            const uint64_t size = kv8_pack(fabsf(x[4 * i]) + fabsf(x[4 * i + 1]), fabsf(x[4 * i + 2]) + fabsf(x[4 * i + 3]));
            const uint64_t d = kv8_mul2(size, off), md = kv8_mul2(size, minus);
            const float2 l02 = kv8_unpack(kv8_fma2(x02, up2, md)), l13 = kv8_unpack(kv8_fma2(x13, up2, md));
            const float2 h02 = kv8_unpack(kv8_fma2(x02, up2, d)), h13 = kv8_unpack(kv8_fma2(x13, up2, d));
            w[i] = kv8_code4(l02.x, l13.x, l02.y, l13.y);
            z[i] = kv8_code4(h02.x, h13.x, h02.y, h13.y);
            differ |= w[i] ^ z[i];
          }
          if (differ) {
            differ = 0u;
#pragma unroll
            for (int i = 0; i < 8; i++) differ |= uint32_t(w[i] != z[i]) << i;
          }
        }
        differ &= on ? me.live : 0u;                                     // (a zero of no row may differ in its sign)
        if (__any_sync(0xffffffffu, differ != 0u)) {
          const int more = __reduce_add_sync(0xffffffffu, __popc(differ));
          if (steps > 1 && later + more <= 32) {
            mine &= ~differ;
#pragma unroll 1
            for (int i = 0; i < 8; i++) {
              const uint32_t m = __ballot_sync(0xffffffffu, differ >> i & 1u);
              if (differ >> i & 1u) sh.later[t >> 5][later + __popc(m & ((1u << lane) - 1u))] = uint32_t(step << 8 | lane << 3 | i);
              later += __popc(m);
            }
          } else {
            const uint32_t again_in = __reduce_or_sync(0xffffffffu, differ);
            float y[32];
            kv8_exact_keys(from, me.row_stride, on ? me.live & again_in : 0u, turned, sh.circle, sh.phase + me.d0 / 2, me.pos0, y);
#pragma unroll
            for (int i = 0; i < 8; i++)
              if (on && (me.live & again_in) >> i & 1u) w[i] = kv8_code4(y[4 * i] * up, y[4 * i + 1] * up, y[4 * i + 2] * up, y[4 * i + 3] * up);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; i++) {
          uint32_t y[2];
          kv8_half4(w[i], y[0], y[1]);
          if (mine >> i & 1u) {
#pragma unroll
            for (int j = 0; j < 2; j++) {
              lo[j] = kv8_min2(lo[j], y[j]);
              hi[j] = kv8_max2(hi[j], y[j]);
            }
          }
        }
      }
      const int group = t / (HD / 4);
      *reinterpret_cast<uint2*>(&sh.lo[buf][group * (HD / 2) + me.d0 / 2]) = make_uint2(lo[0], lo[1]);
      *reinterpret_cast<uint2*>(&sh.hi[buf][group * (HD / 2) + me.d0 / 2]) = make_uint2(hi[0], hi[1]);
      if (busy || again) kv8_put_k<HD>(me, w, me.base + L.k(on ? g : 0), on, again, f);
      f_was = f;
    }
    if (on && th == 0) *exps = int8_t(e);
  }
  if (!V) {
    __syncthreads();
    join_bounds((steps - 1) & 1);
    if (!__syncthreads_or(later)) return;
    if (lane >= later) return;
    // a key of this warp's: the codes in their places, and the bounds (which other warps' keys may reach too)
    const uint32_t what = sh.later[t >> 5][lane];
    const int of = (t & ~31) | int(what >> 3 & 31u), th1 = of % tph, g1 = g0 + (of / tph - hp) + int(what >> 8) * abreast;
    const int d1 = 4 * (th1 % (HD / 4)), p1 = 8 * (th1 / (HD / 4)) + int(what & 7u);
    const T* from = src + int64_t(p1 - me.p0) * me.row_stride + (d1 - me.d0) + int64_t(g1) * head_stride;
    const int e = *reinterpret_cast<const int8_t*>(me.base + L.exps(g1));
    const uint32_t w = kv8_exact_codes(from, turned, sh.circle, sh.phase + d1 / 2, me.pos0 - me.p0 + p1, kv8_exp2i(-e));
    *reinterpret_cast<uint32_t*>(me.base + L.k(g1) + kv8_k_at(HD, p1, d1 >> 4) + (d1 & 15)) = w;
    uint32_t y[2], least = 0u, most = 0u;
    kv8_half4(w, y[0], y[1]);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const float x = __half2float(__ushort_as_half(uint16_t(y[j / 2] >> (16 * (j & 1)))));
      least |= uint32_t(uint8_t(x != x ? -127 : int(floorf(x * 0.25f)))) << (8 * j);
      most |= uint32_t(uint8_t(x != x ? 127 : int(ceilf(x * 0.25f)))) << (8 * j);
    }
    auto join = [](uint32_t* at, uint32_t x, bool up) {
      uint32_t is = *reinterpret_cast<volatile uint32_t*>(at), was;
      do {
        was = is;
        is = atomicCAS(at, was, up ? __vmaxs4(was, x) : __vmins4(was, x));
      } while (is != was);
    };
    uint32_t* at = reinterpret_cast<uint32_t*>(me.base + L.bounds(g1) + d1);
    join(at, least, false);
    join(at + HD / 4, most, true);
  }
}

template <int HD, class T, int NT>
__global__ void __launch_bounds__(NT, NT == 512 ? 1 : 2) k_kv8_append(Kv4 c, Kv4Rows a, Kv8Rot r, const T* k, const T* v,
                                                                                         const T* q) {
  __shared__ Kv8AppendShared<HD, NT> sh;
  const int t = threadIdx.x;
  if (r.on) {
    for (int i = t; i < HD / 2; i += NT) sh.phase[i] = r.phase[i];
    // (lookups that differ by lane, 16 a thread, take 8000 cycles a CTA out of global memory)
    for (int i = t; i < 256; i += NT) sh.circle[i] = kKv8Circle.p[i];
  }
  kv4_dependent();
  if (kv4_check_rows(c, a)) return;
  const int64_t id = int64_t(blockIdx.x) - a.checks, pages = int64_t(a.units) * r.splits * 2;
  if (id >= pages) {
    __syncthreads();
    kv8_rotate_q<HD, T>(c, a, r, sh.circle, sh.phase, q, id - pages);
    return;
  }
  // K first: a CTA of it takes longer (16000 f16 rows, 8 heads of 128: 36 us; K and V by turns: 46)
  const bool is_v = id >= pages / 2;
  const int64_t part = is_v ? id - pages / 2 : id;
  const int P = c.page_len, split = int(part % r.splits);
  Kv4Span sp;
  if (!kv4_span(c, a, int(part / r.splits), &sp, P)) return;
  const Kv8Page L(c);
  const int tph = P * HD / 32, th = t % tph, abreast = NT / tph;      // threads of a head, heads side by side
  Kv8Mine me;
  me.row_stride = a.row_stride;
  me.d0 = is_v ? 2 * (th % (HD / 2)) : 4 * (th % (HD / 4));
  me.p0 = is_v ? 16 * (th / (HD / 2)) : 8 * (th / (HD / 4));
  me.pos0 = sp.p0 + me.p0;
  me.first = sp.first;
  me.last = sp.last;
  me.fresh = sp.first == 0;
  me.live = 0u;
  for (int i = 0; i < (is_v ? 16 : 8); i++)
    if (me.p0 + i >= sp.first && me.p0 + i < sp.last) me.live |= 1u << i;
  const int g = split * r.per * abreast + t / tph;
  const int left = (c.n_kv - split * r.per * abreast + abreast - 1) / abreast, steps = left < r.per ? left : r.per;
  const T* src = (is_v ? v : k) + int64_t(sp.row - sp.first + me.p0) * a.row_stride + me.d0;
  const int page = c.table[int64_t(sp.s) * c.max_pages + sp.p0 / P];
  uint32_t raw[Kv8Raw<T>::kWords];                                    // (on the way while the page is looked up)
  if (is_v) kv8_load<T, true>(me, src + int64_t(g) * a.head_stride, g < c.n_kv, raw);
  else kv8_load<T, false>(me, src + int64_t(g) * a.head_stride, g < c.n_kv, raw);
  if (!is_v && r.on) {
    __syncthreads();   // the phases
    constexpr int kSide = NT / (HD / 2);                               // positions side by side
    const int pair = t % (HD / 2);
    const uint64_t phase = sh.phase[pair], step = phase * kSide;
    int p = sp.first + t / (HD / 2);
    uint64_t turn = phase * uint64_t(uint32_t(sp.p0 + p));
    float* to = kv8_turns + (pair >> 1) * 4 + (pair & 1);
#pragma unroll 4
    for (; p < sp.last; p += kSide, turn += step) {
      const float2 z = kv8_turn_fast(sh.circle, turn);
      to[p * HD] = z.x;
      to[p * HD + 2] = z.y;
    }
    __syncthreads();
  }
  if (page < 0 || page >= c.n_pages || c.refs[page] != 1) {
    if (t == 0) kv4_flag(c, NT_KV4_BAD_PAGE);
    return;
  }
  me.base = c.pool + (int64_t(a.layer) * c.n_pages + page) * c.page_bytes();
  if (is_v) kv8_append_page<HD, T, NT, true>(c, L, me, sh, src, a.head_stride, false, g, abreast, steps, raw);
  else kv8_append_page<HD, T, NT, false>(c, L, me, sh, src, a.head_stride, r.on, g, abreast, steps, raw);
}

// Four values into consecutive elements.
__device__ __forceinline__ void kv8_put4(float* p, float2 a, float2 b) { *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y); }
__device__ __forceinline__ void kv8_put4(__half* p, float2 a, float2 b) {
  const __half2 lo = __floats2half2_rn(a.x, a.y), hi = __floats2half2_rn(b.x, b.y);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}
// Four words of four bytes each, transposed.
__device__ __forceinline__ void kv8_transpose(uint32_t (&w)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[0], w[1], 0x7362);
  const uint32_t c = __byte_perm(w[2], w[3], 0x5140), d = __byte_perm(w[2], w[3], 0x7362);
  w[0] = __byte_perm(a, c, 0x5410);
  w[1] = __byte_perm(a, c, 0x7632);
  w[2] = __byte_perm(b, d, 0x5410);
  w[3] = __byte_perm(b, d, 0x7632);
}

constexpr int kKv8ReadWarps = 4;   // warps of a CTA: each K or V of a (unit, kv head)

template <int HD, class T>
__global__ void __launch_bounds__(32 * kKv8ReadWarps) k_kv8_read(Kv4 c, Kv4Rows a, T* k, T* v) {
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t(blockIdx.x) - a.checks) * kKv8ReadWarps + (threadIdx.x >> 5);   // (below 0: see kv4_check_rows)
  const int g = int(id / 2 % c.n_kv);
  const int64_t u = id / 2 / c.n_kv;
  if (u >= a.units) return;
  kv4_dependent();
  if (kv4_check_rows(c, a)) return;
  Kv4Span sp;
  if (!kv4_span(c, a, int(u), &sp)) return;
  const int page = c.table[int64_t(sp.s) * c.max_pages + sp.p0 / c.page_len];
  if (page < 0 || page >= c.n_pages) {
    if (lane == 0) kv4_flag(c, NT_KV4_BAD_PAGE);
    return;
  }
  const Kv8Page L(c);
  const uint8_t* base = c.pool + (int64_t(a.layer) * c.n_pages + page) * c.page_bytes();
  const int at0 = sp.p0 % c.page_len;                                  // the chunk's place in its page
  const int8_t* exps = reinterpret_cast<const int8_t*>(base + L.exps(g));
  const int64_t row0 = int64_t(sp.row - sp.first) * a.row_stride + int64_t(g) * a.head_stride;
  constexpr int kLanes = HD / 4, kRows = 32 / kLanes;                  // lanes of a row, rows side by side
  const int d = 4 * (lane % kLanes), sub = lane / kLanes;
  auto put = [&](T* to, uint32_t w, float f) {
    float2 x = kv8_value2(w & 0xffffu), y = kv8_value2(w >> 16);
    x.x *= f; x.y *= f; y.x *= f; y.y *= f;
    kv8_put4(to, x, y);
  };
  if (!(id & 1)) {
    // four dimensions a lane, a word
    const uint8_t* from = base + L.k(g) + kv8_k_at(HD, at0, d >> 4) + (d & 15);
    uint32_t w[16 / kRows];
#pragma unroll
    for (int i = 0; i < 16 / kRows; i++) w[i] = *reinterpret_cast<const uint32_t*>(from + kv8_k_at(HD, i * kRows + sub, 0));
    const float f = kv8_exp2i(exps[0]);
#pragma unroll
    for (int i = 0; i < 16 / kRows; i++) {
      const int p = i * kRows + sub;
      if (p >= sp.first && p < sp.last) put(k + row0 + int64_t(p) * a.row_stride + d, w[i], f);
    }
  } else {
    // four dimensions of 16 positions (64 dimensions: of 8), their bytes turned round
    constexpr int kPos = 16 / kRows;
    const uint8_t* from = base + L.v(g) + kv8_v_at(HD, at0 >> 4, d) + kPos * sub;
    uint32_t w[kPos / 4][4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      if (kPos == 16) {
        const uint4 y = *reinterpret_cast<const uint4*>(from + 16 * j);
        w[0][j] = y.x; w[1][j] = y.y; w[2 % (kPos / 4)][j] = y.z; w[3 % (kPos / 4)][j] = y.w;
      } else {
        const uint2 y = *reinterpret_cast<const uint2*>(from + 16 * j);
        w[0][j] = y.x; w[1][j] = y.y;
      }
    }
    const float f = kv8_exp2i(exps[1]);
#pragma unroll
    for (int i = 0; i < kPos / 4; i++) {
      kv8_transpose(w[i]);
#pragma unroll
      for (int b = 0; b < 4; b++) {
        const int p = kPos * sub + 4 * i + b;
        if (p >= sp.first && p < sp.last) put(v + row0 + int64_t(p) * a.row_stride + d, w[i][b], f);
      }
    }
  }
}

// f / (2 pi) modulo 1 as a 64-bit fraction, to its last bit or two (|f| up to 2^20).
static uint64_t kv8_phase(double f) {
  constexpr double h = 0.15915494309189535, l = -9.839338337591243e-18;   // 1 / (2 pi) as a sum of two doubles
  const double a = std::fabs(f), p = a * h, e = std::fma(a, h, -p) + a * l;   // p + e: within 2^-80 or so
  const double frac = p - std::floor(p);                                    // exact (not so below zero: the sign comes last)
  // the fraction in two exact steps of 32 bits
  const double upper = std::floor(frac * 4294967296.0), lower = (frac * 4294967296.0 - upper) * 4294967296.0;
  const double rest = std::nearbyint(e * 18446744073709551616.0);          // |e| < 2^-33: below 2^31
  const uint64_t turn = (uint64_t(upper) << 32) + uint64_t(int64_t(std::nearbyint(lower)) + int64_t(rest));
  return f < 0 ? 0 - turn : turn;
}

// CTA of an append: the threads of one page and kv head, 256 at least (then several heads side by side).
static int kv8_append_threads(const Kv4& k) { return k.page_len * k.hd / 32 > 256 ? 512 : 256; }

template <int HD, class T, int NT>
static cudaError_t kv8_launch_append(const Kv4& k, const Kv4Rows& a, const Kv8Rot& r, unsigned grid, cudaStream_t s, const void* pk,
                                     const void* pv, const void* pq) {
  static const KernelSetup setup = kernel_setup(k_kv8_append<HD, T, NT>, 128 * HD * 4);
  if (setup.err != cudaSuccess) return setup.err;
  return kv4_launch_smem(k_kv8_append<HD, T, NT>, grid, unsigned(NT), r.on ? size_t(k.page_len) * HD * 4 : 0, s, k, a, r,
                         static_cast<const T*>(pk), static_cast<const T*>(pv), static_cast<const T*>(pq));
}
template <class T>
static cudaError_t kv8_launch_append(const Kv4& k, const Kv4Rows& a, const Kv8Rot& r, unsigned grid, cudaStream_t s, const void* pk,
                                     const void* pv, const void* pq) {
  if (k.hd == 64) return kv8_launch_append<64, T, 256>(k, a, r, grid, s, pk, pv, pq);
  return kv8_append_threads(k) == 512 ? kv8_launch_append<128, T, 512>(k, a, r, grid, s, pk, pv, pq)
                                      : kv8_launch_append<128, T, 256>(k, a, r, grid, s, pk, pv, pq);
}

}  // namespace nt

using namespace nt;

extern "C" {

nt_status nt_kv8_pool_bytes(const nt_kv8_cache* c, size_t* page_bytes, size_t* pool_bytes) {
  Kv4 k;
  const nt_status st = kv8_check(c, "nt_kv8_pool_bytes", false, &k);
  if (st) return st;
  if (page_bytes) *page_bytes = size_t(k.page_bytes());
  if (pool_bytes) *pool_bytes = size_t(k.page_bytes()) * size_t(k.n_pages) * size_t(k.n_layers);
  return NT_OK;
}

nt_status nt_kv8_workspace_bytes(const nt_kv8_cache* c, int32_t n_heads, int32_t n, size_t* bytes) {
  Kv4 k;
  const nt_status st = kv8_check(c, "nt_kv8_workspace_bytes", false, &k);
  if (st) return st;
  if (!bytes) return fail(NT_E_INVAL, "nt_kv8_workspace_bytes: NULL argument");
  if (n < 0 || n_heads < 1) return fail(NT_E_INVAL, "nt_kv8_workspace_bytes: n or n_heads out of range");
  if (n_heads % k.n_kv) return fail(NT_E_INVAL, "nt_kv8_workspace_bytes: n_heads must be a multiple of n_kv_heads");
  n = n < kKv4MaxSeqs ? n : kKv4MaxSeqs;   // (no call takes more, and the sizes fit 64 bits)
  const size_t w[3] = {kv4_ws(k, n).bytes, kv8_select_ws_bytes(k, n), kv8_attn_ws_bytes(k.hd)};
  *bytes = w[0] > w[1] ? w[0] : w[1];
  if (w[2] > *bytes) *bytes = w[2];
  return NT_OK;
}

nt_status nt_kv8_extend(const nt_kv8_cache* c, int32_t n, const int32_t* dev_seq, const int32_t* dev_count,
                        void* dev_workspace, size_t workspace_bytes, void* stream) {
  Kv4 k;
  const nt_status st = kv8_check(c, "nt_kv8_extend", true, &k);
  return st ? st : kv4_extend("nt_kv8_extend", k, n, dev_seq, dev_count, dev_workspace, workspace_bytes, stream);
}

nt_status nt_kv8_fork(const nt_kv8_cache* c, int32_t n, const int32_t* dev_src, const int32_t* dev_dst,
                      const int32_t* dev_keep, void* dev_workspace, size_t workspace_bytes, void* stream) {
  Kv4 k;
  const nt_status st = kv8_check(c, "nt_kv8_fork", true, &k);
  return st ? st : kv4_fork("nt_kv8_fork", k, n, dev_src, dev_dst, dev_keep, dev_workspace, workspace_bytes, stream);
}

nt_status nt_kv8_free(const nt_kv8_cache* c, int32_t n, const int32_t* dev_seq, const int32_t* dev_keep, void* stream) {
  Kv4 k;
  const nt_status st = kv8_check(c, "nt_kv8_free", true, &k);
  return st ? st : kv4_free("nt_kv8_free", k, n, dev_seq, dev_keep, stream);
}

nt_status nt_kv8_copy_pages(const nt_kv8_cache* c, int32_t n, const int32_t* dev_src, const int32_t* dev_dst,
                            void* stream) {
  Kv4 k;
  const nt_status st = kv8_check(c, "nt_kv8_copy_pages", true, &k);
  return st ? st : kv4_copy_pages("nt_kv8_copy_pages", k, n, dev_src, dev_dst, stream);
}

nt_status nt_kv8_compact(const nt_kv8_cache* c, int32_t* dev_table_out, int32_t* dev_refs_out, int32_t* dev_live,
                         void* dev_workspace, size_t workspace_bytes, void* stream) {
  Kv4 k;
  const nt_status st = kv8_check(c, "nt_kv8_compact", true, &k);
  return st ? st : kv4_compact("nt_kv8_compact", k, dev_table_out, dev_refs_out, dev_live, dev_workspace, workspace_bytes, stream);
}

nt_status nt_kv8_append(const nt_kv8_cache* c, int32_t layer, int32_t n, const int32_t* dev_seq,
                        const int32_t* dev_begin, int32_t n_rows, nt_qtype type, const void* dev_k, const void* dev_v,
                        int64_t row_stride, int64_t head_stride, const double* freq, int32_t n_heads, const void* dev_q,
                        int64_t q_stride, float* dev_q_out, int64_t q_out_stride, void* stream) {
  const char* who = "nt_kv8_append";
  auto bad = [&](const char* what) { return fail(NT_E_INVAL, std::string(who) + ": " + what); };
  Kv4 k;
  nt_status st = kv8_check(c, who, true, &k);
  if (st) return st;
  const Kv4Rows a{layer, n, n_rows, kv4_units(n, n_rows, dev_begin, k.page_len), kv4_checks(n, n_rows, dev_begin), dev_seq,
                  dev_begin, row_stride, head_stride};
  st = kv4_rows_check(who, k, a, type, dev_k, dev_v);
  if (!st && n > k.max_seqs) st = bad("n above max_seqs");
  if (!st) st = kv4_array_check(k, who, dev_seq, n, true, nullptr, 0);
  if (!st) st = kv4_array_check(k, who, dev_begin, int64_t(n) + 1, true, nullptr, 0);
  if (st) return st;
  Kv8Rot r{};
  if (freq) {
    r.on = 1;
    for (int i = 0; i < k.hd / 2; i++) {
      if (!(std::fabs(freq[i]) <= 1048576.0)) return bad("a frequency is not finite or above 2^20");
      r.phase[i] = kv8_phase(freq[i]);
    }
  }
  const int64_t es = type == NT_F32 ? 4 : 2, most = int64_t(1) << 40;
  if (dev_q) {
    if (!freq) return bad("q without frequencies");
    if (n_heads < 1 || n_heads > 65535) return bad("n_heads outside [1, 65535]");
    const int64_t row = int64_t(n_heads) * k.hd;
    if (!kv4_aligned(dev_q, 16) || !kv4_aligned(dev_q_out, 16)) return bad("q or q_out is NULL or not 16-byte aligned");
    if (q_stride < row || q_out_stride < row || q_stride * es % 16 || q_out_stride % 4 || q_stride > most || q_out_stride > most)
      return bad("q strides must be multiples of 16 bytes and at least n_heads * head_dim");
    r.heads = n_heads;
    r.q_stride = q_stride;
    r.out_stride = q_out_stride;
    r.out = dev_q_out;
  } else if (dev_q_out) {
    return bad("q_out without q");
  }
  if (n == 0 || n_rows == 0) return NT_OK;
  const int64_t bytes = kv4_rows_bytes(k, a, type);
  if (bytes < 0) return bad("the strides are too large");
  if (kv4_meets_cache(k, dev_k, bytes) || kv4_meets_cache(k, dev_v, bytes)) return bad("k or v overlaps the cache");
  int64_t q_ctas = 0;
  if (dev_q) {
    if (double(n_rows) * double(q_stride > q_out_stride ? q_stride : q_out_stride) > 1e17) return bad("the strides are too large");
    const int64_t row = int64_t(n_heads) * k.hd, qb = ((n_rows - 1) * q_stride + row) * es, ob = ((n_rows - 1) * q_out_stride + row) * 4;
    const bool in_place = static_cast<const void*>(dev_q_out) == dev_q && type == NT_F32 && q_stride == q_out_stride;
    if ((!in_place && kv4_overlap(dev_q_out, ob, dev_q, qb)) || kv4_overlap(dev_q_out, ob, dev_k, bytes) ||
        kv4_overlap(dev_q_out, ob, dev_v, bytes) || kv4_meets_cache(k, dev_q_out, ob) || kv4_meets_cache(k, dev_q, qb) ||
        kv4_overlap(dev_seq, dev_seq ? int64_t(n) * 4 : 0, dev_q_out, ob) ||
        kv4_overlap(dev_begin, dev_begin ? int64_t(n) * 4 + 4 : 0, dev_q_out, ob))
      return bad("q_out overlaps another buffer");
    auto with = [&](int heads) { return int64_t(n_rows) * ((n_heads + heads - 1) / heads); };
    r.q_heads = with(16) >= kKv8QWarps16 ? 16 : with(8) >= kKv8QWarps8 ? 8 : 4;
    const int64_t warps = with(r.q_heads), of_cta = kv8_append_threads(k) / 32;
    q_ctas = (warps + of_cta - 1) / of_cta;
  }
  const int threads = kv8_append_threads(k), abreast = threads * 32 / (k.page_len * k.hd), steps = (k.n_kv + abreast - 1) / abreast;
  const int64_t each = (int64_t(a.units) * 2 * steps * threads / 256 + kKv8AppendCtas - 1) / kKv8AppendCtas;
  r.splits = each >= steps ? 1 : int32_t((steps + each - 1) / each);
  r.per = (steps + r.splits - 1) / r.splits;
  r.splits = (steps + r.per - 1) / r.per;
  const int64_t grid = int64_t(a.units) * r.splits * 2 + a.checks + q_ctas;
  if (grid > 0x7fffffffLL) return bad("too many rows for one call");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == NT_F32 ? kv8_launch_append<float>(k, a, r, unsigned(grid), s, dev_k, dev_v, dev_q)
                                       : kv8_launch_append<__half>(k, a, r, unsigned(grid), s, dev_k, dev_v, dev_q);
  if (e != cudaSuccess) return cuda_fail(e, who);
  if (dev_seq && n > 1) NT_CUDA(kv4_launch_listed_twice(k, n, dev_seq, s));
  return NT_OK;
}

nt_status nt_kv8_read(const nt_kv8_cache* c, int32_t layer, int32_t n, const int32_t* dev_seq, const int32_t* dev_begin,
                      int32_t n_rows, nt_qtype type, void* dev_k, void* dev_v, int64_t row_stride, int64_t head_stride,
                      void* stream) {
  const char* who = "nt_kv8_read";
  auto bad = [&](const char* what) { return fail(NT_E_INVAL, std::string(who) + ": " + what); };
  Kv4 k;
  nt_status st = kv8_check(c, who, true, &k);
  if (st) return st;
  const Kv4Rows a{layer, n, n_rows, kv4_units(n, n_rows, dev_begin), kv4_checks(n, n_rows, dev_begin), dev_seq, dev_begin, row_stride,
                  head_stride};
  st = kv4_rows_check(who, k, a, type, dev_k, dev_v);
  if (!st) st = kv4_array_check(k, who, dev_seq, n, true, nullptr, 0);
  if (!st) st = kv4_array_check(k, who, dev_begin, int64_t(n) + 1, true, nullptr, 0);
  if (st || n == 0 || n_rows == 0) return st;
  const int64_t bytes = kv4_rows_bytes(k, a, type), es = type == NT_F32 ? 4 : 2;
  if (bytes < 0) return bad("the strides are too large");
  const int64_t apart = static_cast<char*>(dev_v) - static_cast<char*>(dev_k);
  if (kv4_rows_meet(k, a, es, 0, true) || (kv4_overlap(dev_k, bytes, dev_v, bytes) && kv4_rows_meet(k, a, es, apart, false)))
    return bad("rows of the outputs overlap");
  if (kv4_meets_cache(k, dev_k, bytes) || kv4_meets_cache(k, dev_v, bytes) ||
      kv4_overlap(dev_seq, int64_t(n) * 4, dev_k, bytes) || kv4_overlap(dev_seq, int64_t(n) * 4, dev_v, bytes) ||
      kv4_overlap(dev_begin, int64_t(n) * 4 + 4, dev_k, bytes) || kv4_overlap(dev_begin, int64_t(n) * 4 + 4, dev_v, bytes))
    return bad("an output overlaps another buffer");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned nt = 32u * kKv8ReadWarps, gr = unsigned((int64_t(a.units) * k.n_kv * 2 + kKv8ReadWarps - 1) / kKv8ReadWarps + a.checks);
  if (type == NT_F32) {
    float *pk = static_cast<float*>(dev_k), *pv = static_cast<float*>(dev_v);
    NT_CUDA(k.hd == 64 ? kv4_launch(k_kv8_read<64, float>, gr, nt, s, k, a, pk, pv) : kv4_launch(k_kv8_read<128, float>, gr, nt, s, k, a, pk, pv));
  } else {
    __half *pk = static_cast<__half*>(dev_k), *pv = static_cast<__half*>(dev_v);
    NT_CUDA(k.hd == 64 ? kv4_launch(k_kv8_read<64, __half>, gr, nt, s, k, a, pk, pv) : kv4_launch(k_kv8_read<128, __half>, gr, nt, s, k, a, pk, pv));
  }
  return NT_OK;
}

}  // extern "C"
