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

struct Kv8Circle {
  float c[256], cl[256], s[256], sl[256];
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
    t.c[i] = float(c);
    t.cl[i] = float(c - double(t.c[i]));
    t.s[i] = float(s);
    t.sl[i] = float(s - double(t.s[i]));
  }
  return t;
}
__device__ constexpr Kv8Circle kKv8Circle = kv8_circle();

struct Kv8Turn {
  float c, cl, s, sl;   // cos, sin: the sums of two terms
};
// a + b in two terms (a in hi already: hi = a + b rounded)
__device__ __forceinline__ float kv8_rest(float a, float b, float hi) {
  const float bb = __fsub_rn(hi, a);
  return __fadd_rn(__fsub_rn(a, __fsub_rn(hi, bb)), __fsub_rn(b, bb));
}
__device__ __forceinline__ Kv8Turn kv8_turn(uint64_t phase, int pos) {
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
  const float C = kKv8Circle.c[i], Cl = kKv8Circle.cl[i], S = kKv8Circle.s[i], Sl = kKv8Circle.sl[i];
  auto times = [](float x, float xl, float y, float yl, float& p) {          // (x + xl) (y + yl) = p + the rest
    p = __fmul_rn(x, y);
    return __fadd_rn(__fmaf_rn(x, y, -p), __fmaf_rn(x, yl, __fmul_rn(xl, y)));
  };
  Kv8Turn t;
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
__device__ __forceinline__ void kv8_rotate(const Kv8Turn& t, float& a, float& b) {
  const float x = kv8_dot2(a, t.c, t.cl, b, -t.s, -t.sl);
  b = kv8_dot2(a, t.s, t.sl, b, t.c, t.cl);
  a = x;
}

// ------------------------------------------------------------ append, read --
//
// A CTA handles K or V of one page of one sequence and kv head, the rows that fall on
// its positions: the page's exponent needs all of them before the first code.

struct Kv8Rot {
  uint64_t phase[64];   // turns per position, as 64-bit fractions
  int32_t on, heads;
  int64_t q_stride, out_stride;
  float* out;
};

constexpr int kKv8RowThreads = 256;
constexpr int kKv8QHeads = 4;   // heads that a warp rotates

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
__device__ __forceinline__ void kv8_rotate_q(const Kv4& c, const Kv4Rows& a, const Kv8Rot& r, const uint64_t* phase, const T* q,
                                             int64_t id) {
  constexpr int kLanes = HD / 4;           // of a head
  const int lane = threadIdx.x & 31, groups = (r.heads + kKv8QHeads - 1) / kKv8QHeads;
  const int64_t unit = id * (kKv8RowThreads / 32) + (threadIdx.x >> 5);
  if (unit >= int64_t(a.n_rows) * groups) return;
  const int row = int(unit / groups), h0 = int(unit % groups) * kKv8QHeads;
  const int pos = kv8_row_pos(c, a, row);
  if (pos < 0) return;
  const int i = lane % kLanes;
  const Kv8Turn t0 = kv8_turn(phase[2 * i], pos), t1 = kv8_turn(phase[2 * i + 1], pos);
#pragma unroll
  for (int y = 0; y < kKv8QHeads; y += 32 / kLanes) {
    const int h = h0 + y + lane / kLanes;
    if (h >= r.heads) break;
    float4 x = Kv8Quad<T>::get(q + int64_t(row) * r.q_stride + h * HD + 4 * i);
    kv8_rotate(t0, x.x, x.y);
    kv8_rotate(t1, x.z, x.w);
    *reinterpret_cast<float4*>(r.out + int64_t(row) * r.out_stride + h * HD + 4 * i) = x;
  }
}

template <int HD, class T>
__global__ void __launch_bounds__(kKv8RowThreads) k_kv8_append(Kv4 c, Kv4Rows a, Kv8Rot r, const T* k, const T* v, const T* q) {
  constexpr int NT = kKv8RowThreads, kQuads = HD / 4, kStride = HD + 4;
  extern __shared__ __align__(16) float kv8_rows[];   // [page_len][kStride]
  __shared__ uint64_t s_phase[HD / 2];
  __shared__ float s_top[NT / 32];
  const int t = threadIdx.x;
  for (int i = t; i < HD / 2; i += NT) s_phase[i] = r.phase[i];
  __syncthreads();
  kv4_dependent();
  if (kv4_check_rows(c, a)) return;
  const int64_t id = int64_t(blockIdx.x) - a.checks, pages = int64_t(a.units) * c.n_kv * 2;
  if (id >= pages) {
    kv8_rotate_q<HD, T>(c, a, r, s_phase, q, id - pages);
    return;
  }
  const bool is_v = id & 1;
  const int g = int(id / 2 % c.n_kv);
  Kv4Span sp;
  if (!kv4_span(c, a, int(id / 2 / c.n_kv), &sp, c.page_len)) return;
  const int page = c.table[int64_t(sp.s) * c.max_pages + sp.p0 / c.page_len];
  if (page < 0 || page >= c.n_pages || c.refs[page] != 1) {
    if (t == 0) kv4_flag(c, NT_KV4_BAD_PAGE);
    return;
  }
  const Kv8Page L(c);
  uint8_t* base = c.pool + (int64_t(a.layer) * c.n_pages + page) * c.page_bytes();
  // ---- the rows, rotated, into shared memory; their largest magnitude
  const T* src = (is_v ? v : k) + int64_t(sp.row - sp.first) * a.row_stride + int64_t(g) * a.head_stride;   // of position 0
  float top = 0.f;
  const int quad = t % kQuads;
  for (int p = sp.first + t / kQuads; p < sp.last; p += NT / kQuads) {
    float4 x = Kv8Quad<T>::get(src + int64_t(p) * a.row_stride + 4 * quad);
    if (!is_v && r.on) {
      kv8_rotate(kv8_turn(s_phase[2 * quad], sp.p0 + p), x.x, x.y);
      kv8_rotate(kv8_turn(s_phase[2 * quad + 1], sp.p0 + p), x.z, x.w);
    }
    *reinterpret_cast<float4*>(kv8_rows + p * kStride + 4 * quad) = x;
    auto size = [](float y) { return kv8_held(y) ? fabsf(y) : 0.f; };
    top = fmaxf(top, fmaxf(fmaxf(size(x.x), size(x.y)), fmaxf(size(x.z), size(x.w))));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((t & 31) == 0) s_top[t >> 5] = top;
  int8_t* exps = reinterpret_cast<int8_t*>(base + L.exps(g)) + is_v;
  const bool fresh = sp.first == 0;
  const int was = fresh ? kKv8MinExp : *exps;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / 32; i++) top = fmaxf(top, s_top[i]);
  int e = kv8_exponent(top);
  if (e < was) e = was;
  const float up = kv8_exp2i(-e);
  const int less = e - was;                                            // exponents that older codes are rounded for
  const bool again = !fresh && less > 0;
  const float f = kv8_exp2i(less > 126 ? -126 : -less);                // (from 2^-20 on every code is rounded to zero)
  if (!is_v) {
    uint8_t* to = base + L.k(g);
    for (int i = t; i < sp.last * (HD / 16); i += NT) {
      const int p = i % sp.last, ch = i / sp.last;
      uint4* at = reinterpret_cast<uint4*>(to + kv8_k_at(HD, p, ch));
      if (p < sp.first) {
        if (again) *at = kv8_again(*at, f);
        continue;
      }
      uint32_t w[4];
#pragma unroll
      for (int y = 0; y < 4; y++) {
        const float4 x = *reinterpret_cast<const float4*>(kv8_rows + p * kStride + 16 * ch + 4 * y);
        w[y] = kv8_code4(kv8_scaled(x.x, up), kv8_scaled(x.y, up), kv8_scaled(x.z, up), kv8_scaled(x.w, up));
      }
      *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
    // bounds: the least and the largest value round to the least and the largest code
    if (t < HD) {
      float least = INFINITY, most = -INFINITY;
      bool nan = false;
      for (int p = sp.first; p < sp.last; p++) {
        const float x = kv8_rows[p * kStride + t];
        nan |= !kv8_held(x);
        least = fminf(least, x);
        most = fmaxf(most, x);
      }
      const float2 y = kv8_value2(kv8_code2(least * up, most * up));
      int lo = nan ? -127 : int(floorf(y.x * 0.25f)), hi = nan ? 127 : int(ceilf(y.y * 0.25f));
      int8_t* b = reinterpret_cast<int8_t*>(base + L.bounds(g)) + t;
      if (!fresh) {
        int lo0 = b[0], hi0 = b[HD];
        if (lo0 != -127) lo0 = int(floorf(lo0 * f));
        if (hi0 != 127) hi0 = int(ceilf(hi0 * f));
        lo = lo0 < lo ? lo0 : lo;
        hi = hi0 > hi ? hi0 : hi;
      }
      b[0] = int8_t(lo);
      b[HD] = int8_t(hi);
    }
  } else {
    uint8_t* to = base + L.v(g);
    const int tc0 = again ? 0 : sp.first / 16, tcs = (sp.last + 15) / 16 - tc0;
    for (int i = t; i < tcs * HD; i += NT) {
      const int tc = tc0 + i / HD, d = i % HD, p0 = 16 * tc;
      uint4* at = reinterpret_cast<uint4*>(to + kv8_v_at(HD, tc, d));
      uint4 old = make_uint4(0u, 0u, 0u, 0u);
      if (p0 < sp.first || p0 + 16 > sp.last) old = *at;
      uint32_t w[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
      for (int y = 0; y < 4; y++) {
        const uint32_t kept = again ? kv8_again(w[y], f) : w[y];
        uint32_t mine = 0u, mask = 0u, held = 0u;                      // the word's new bytes, and those of older positions
        float x[4];
#pragma unroll
        for (int b = 0; b < 4; b++) {
          const int p = p0 + 4 * y + b;
          const bool live = p >= sp.first && p < sp.last;
          x[b] = live ? kv8_scaled(kv8_rows[p * kStride + d], up) : 0.f;
          if (live) mask |= 0xffu << (8 * b);
          if (p < sp.first) held |= 0xffu << (8 * b);
        }
        mine = kv8_code4(x[0], x[1], x[2], x[3]);
        w[y] = (mine & mask) | (kept & held) | (w[y] & ~(mask | held));
      }
      *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  if (t == 0) *exps = int8_t(e);
}

__device__ __forceinline__ void kv8_put(float* p, float x) { *p = x; }
__device__ __forceinline__ void kv8_put(__half* p, float x) { *p = __float2half_rn(x); }

template <int HD, class T>
__global__ void __launch_bounds__(kKv8RowThreads) k_kv8_read(Kv4 c, Kv4Rows a, T* k, T* v) {
  constexpr int NT = kKv8RowThreads;
  const int t = threadIdx.x;
  kv4_dependent();
  if (kv4_check_rows(c, a)) return;
  const int64_t id = int64_t(blockIdx.x) - a.checks;
  const bool is_v = id & 1;
  const int g = int(id / 2 % c.n_kv);
  Kv4Span sp;
  if (!kv4_span(c, a, int(id / 2 / c.n_kv), &sp, c.page_len)) return;
  const int page = c.table[int64_t(sp.s) * c.max_pages + sp.p0 / c.page_len];
  if (page < 0 || page >= c.n_pages) {
    if (t == 0) kv4_flag(c, NT_KV4_BAD_PAGE);
    return;
  }
  const Kv8Page L(c);
  const uint8_t* base = c.pool + (int64_t(a.layer) * c.n_pages + page) * c.page_bytes();
  const float f = kv8_exp2i(reinterpret_cast<const int8_t*>(base + L.exps(g))[is_v]);
  T* to = (is_v ? v : k) + int64_t(sp.row - sp.first) * a.row_stride + int64_t(g) * a.head_stride;   // of position 0
  if (!is_v) {
    const uint8_t* from = base + L.k(g);
    for (int i = t; i < (sp.last - sp.first) * (HD / 16); i += NT) {
      const int p = sp.first + i / (HD / 16), ch = i % (HD / 16);
      const uint4 w = *reinterpret_cast<const uint4*>(from + kv8_k_at(HD, p, ch));
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int y = 0; y < 8; y++) {
        const float2 x = kv8_value2(u[y >> 1] >> (16 * (y & 1)));
        T* at = to + int64_t(p) * a.row_stride + 16 * ch + 2 * y;
        kv8_put(at, x.x * f);
        kv8_put(at + 1, x.y * f);
      }
    }
  } else {
    const uint8_t* from = base + L.v(g);
    const int tc0 = sp.first / 16, tcs = (sp.last + 15) / 16 - tc0;
    for (int i = t; i < tcs * HD; i += NT) {
      const int tc = tc0 + i / HD, d = i % HD;
      const uint4 w = *reinterpret_cast<const uint4*>(from + kv8_v_at(HD, tc, d));
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int y = 0; y < 16; y++) {
        const int p = 16 * tc + y;
        if (p < sp.first || p >= sp.last) continue;
        const float2 x = kv8_value2(u[y >> 2] >> (16 * (y >> 1 & 1)));
        kv8_put(to + int64_t(p) * a.row_stride + d, (y & 1 ? x.y : x.x) * f);
      }
    }
  }
}

// f / (2 pi) modulo 1 as a 64-bit fraction, to its last bit or two (|f| up to 2^20).
static uint64_t kv8_phase(double f) {
  constexpr double h = 0.15915494309189535, l = -9.839338337591243e-18;   // 1 / (2 pi) as a sum of two doubles
  const double p = f * h, e = std::fma(f, h, -p) + f * l;                   // p + e: within 2^-80 or so
  const double whole = std::floor(p), frac = p - whole;                    // exact
  // the fraction in two exact steps of 32 bits
  const double a = std::floor(frac * 4294967296.0), b = (frac * 4294967296.0 - a) * 4294967296.0;
  const double rest = std::nearbyint(e * 18446744073709551616.0);          // |e| < 2^-33: below 2^31
  return (uint64_t(a) << 32) + uint64_t(int64_t(std::nearbyint(b)) + int64_t(rest));
}

template <int HD, class T>
static cudaError_t kv8_launch_append(const Kv4& k, const Kv4Rows& a, const Kv8Rot& r, unsigned grid, cudaStream_t s, const void* pk,
                                     const void* pv, const void* pq) {
  static const KernelSetup setup = kernel_setup(k_kv8_append<HD, T>, 128 * (HD + 4) * 4);
  if (setup.err != cudaSuccess) return setup.err;
  return kv4_launch_smem(k_kv8_append<HD, T>, grid, unsigned(kKv8RowThreads), size_t(k.page_len) * (HD + 4) * 4, s, k, a, r,
                         static_cast<const T*>(pk), static_cast<const T*>(pv), static_cast<const T*>(pq));
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
  const size_t w[3] = {kv4_ws(k, n).bytes, kv8_select_ws_bytes(k, n), kv8_attn_ws_bytes(n_heads, k.n_kv, k.hd)};
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
    const int64_t row = int64_t(n_heads) * k.hd, qb = ((n_rows - 1) * q_stride + row) * es, ob = ((n_rows - 1) * q_out_stride + row) * 4;
    if (double(n_rows) * double(q_stride > q_out_stride ? q_stride : q_out_stride) > 1e17) return bad("the strides are too large");
    const bool in_place = static_cast<const void*>(dev_q_out) == dev_q && type == NT_F32 && q_stride == q_out_stride;
    if ((!in_place && kv4_overlap(dev_q_out, ob, dev_q, qb)) || kv4_overlap(dev_q_out, ob, dev_k, bytes) ||
        kv4_overlap(dev_q_out, ob, dev_v, bytes) || kv4_meets_cache(k, dev_q_out, ob) || kv4_meets_cache(k, dev_q, qb) ||
        kv4_overlap(dev_seq, dev_seq ? int64_t(n) * 4 : 0, dev_q_out, ob) ||
        kv4_overlap(dev_begin, dev_begin ? int64_t(n) * 4 + 4 : 0, dev_q_out, ob))
      return bad("q_out overlaps another buffer");
    const int64_t warps = int64_t(n_rows) * ((n_heads + kKv8QHeads - 1) / kKv8QHeads);
    q_ctas = (warps + kKv8RowThreads / 32 - 1) / (kKv8RowThreads / 32);
  }
  const int64_t grid = int64_t(a.units) * k.n_kv * 2 + a.checks + q_ctas;
  if (grid > 0x7fffffffLL) return bad("too many rows for one call");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (type == NT_F32)
    e = k.hd == 64 ? kv8_launch_append<64, float>(k, a, r, unsigned(grid), s, dev_k, dev_v, dev_q)
                   : kv8_launch_append<128, float>(k, a, r, unsigned(grid), s, dev_k, dev_v, dev_q);
  else
    e = k.hd == 64 ? kv8_launch_append<64, __half>(k, a, r, unsigned(grid), s, dev_k, dev_v, dev_q)
                   : kv8_launch_append<128, __half>(k, a, r, unsigned(grid), s, dev_k, dev_v, dev_q);
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
  const Kv4Rows a{layer, n, n_rows, kv4_units(n, n_rows, dev_begin, k.page_len), kv4_checks(n, n_rows, dev_begin), dev_seq,
                  dev_begin, row_stride, head_stride};
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
  const int64_t grid = int64_t(a.units) * k.n_kv * 2 + a.checks;
  if (grid > 0x7fffffffLL) return bad("too many rows for one call");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned nt = kKv8RowThreads, gr = unsigned(grid);
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
