// nt_kv4.cu -- the paged 4-bit K/V cache: rows into and out of it, and the
// operators on its pages (include/nt.h documents each).
#include "nt_kv4.cuh"

namespace nt {

nt_status kv4_check(const nt_kv4_cache* c, const char* who, bool pointers, Kv4* k) {
  auto bad = [&](const char* what) { return fail(NT_E_INVAL, std::string(who) + ": " + what); };
  if (!c) return bad("NULL cache");
  if (c->n_layers < 1 || c->n_layers > 65535) return bad("n_layers outside [1, 65535]");
  if (c->n_kv_heads < 1 || c->n_kv_heads > 65535) return bad("n_kv_heads outside [1, 65535]");
  if (c->page_len < 16 || c->page_len > 256 || c->page_len % 16) return bad("page_len must be a multiple of 16, 16..256");
  if (c->n_pages < 1) return bad("n_pages must be positive");
  if (c->max_seqs < 1 || c->max_seqs > kKv4MaxSeqs) return bad("max_seqs outside [1, 65536]");
  if (c->max_pages < 1 || int64_t(c->max_pages) * c->page_len > 0x7fffffffLL - 255)
    return bad("max_pages must be positive and max_pages * page_len at most 2^31 - 256");
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(NT_E_UNSUPPORTED, std::string(who) + ": head_dim must be 64 or 128");
  *k = Kv4{c->n_layers, c->n_kv_heads, c->head_dim, c->page_len, c->n_pages, c->max_seqs, c->max_pages,
           static_cast<uint8_t*>(c->pool), c->table, c->len, c->refs, c->error};
  // every byte offset into the pool fits 62 bits
  if (double(k->page_bytes()) * c->n_pages * c->n_layers > 4e18) return bad("the pool is too large");
  if (pointers) {
    if (!kv4_aligned(c->pool, 16)) return bad("pool is NULL or not 16-byte aligned");
    if (!kv4_aligned(c->table, 4) || !kv4_aligned(c->len, 4) || !kv4_aligned(c->refs, 4) || !kv4_aligned(c->error, 4))
      return bad("table, len, refs or error is NULL or not 4-byte aligned");
  }
  return NT_OK;
}

bool kv4_meets_cache(const Kv4& k, const void* p, int64_t bytes) {
  return kv4_overlap(p, bytes, k.pool, k.page_bytes() * k.n_pages * k.n_layers) ||
         kv4_overlap(p, bytes, k.table, int64_t(k.max_seqs) * k.max_pages * 4) ||
         kv4_overlap(p, bytes, k.len, int64_t(k.max_seqs) * 4) || kv4_overlap(p, bytes, k.refs, int64_t(k.n_pages) * 4) ||
         kv4_overlap(p, bytes, k.error, 4);
}

// ------------------------------------------------------------ append, read --
//
// A warp handles K or V of one chunk of one sequence and kv head: the rows that
// fall on its 16 positions.  Both kernels move bytes: a position's K and V are 2 hd
// source elements and 9/8 hd bytes of cache.
//
// append: a lane takes whole blocks of 32 values (the second 16 bytes of a sector
// come from L1), so that maxima and scales need no exchange, a scale is worked out once, and
// three instructions a value are left; the codes cross to the chunk's order in
// shared memory.  (With the chunk's own order in registers, 8 values of a block a lane,
// the scales, worked out 4 and 8 times over, took most of the time: 64.7 us for
// 2 x 20011 f16 rows of 8 heads of 128.)
// read: a lane's words give values that lie side by side in a row across the lanes.

// Every kernel here is launched so that it may start while the one before it in the
// stream ends, and lets the next one start: it touches memory only after that one has
// ended and its writes are visible.
__device__ __forceinline__ void kv4_dependent() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
}
template <class K, class... A>
static cudaError_t kv4_launch_smem(K kern, unsigned grid, unsigned block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
template <class K, class... A>
static cudaError_t kv4_launch(K kern, unsigned grid, unsigned block, cudaStream_t s, A... args) {
  return kv4_launch_smem(kern, grid, block, 0, s, args...);
}

struct Kv4Rows {
  int32_t layer, n, n_rows, units, checks;
  const int32_t* seq;
  const int32_t* begin;
  int64_t row_stride, head_stride;
};

// What a warp works on: positions [first, last) of the chunk at position p0 of
// sequence s are rows of the call, position first's row is `row`.
struct Kv4Span {
  int s, p0, first, last, row;
};

// Flags entries whose rows do not all lie within the call's: their units may be none of the call's.  CTAs of their own
// do it, the grid's first a.checks, so that no warp with rows waits for it.  (16 tokens and 2 x 20011
// f16 rows stored and read back, 5.04 and 71.0 us without: so 5.16 and 71.2; by the warps with rows, at their start or
// end, 5.16 to 5.72 and 71.5 to 75.0.)  Without `begin` there is one such CTA where there
// are more entries than rows.
constexpr int kKv4CheckEntries = 1024;   // of a CTA
__device__ __forceinline__ bool kv4_check_rows(const Kv4& c, const Kv4Rows& a) {
  if (int(blockIdx.x) >= a.checks) return false;
  bool bad = !a.begin;
  const int e1 = (int(blockIdx.x) + 1) * kKv4CheckEntries;   // (2^25 entries at most)
  if (a.begin)
    for (int i = e1 - kKv4CheckEntries + int(threadIdx.x); i < e1 && i < a.n; i += blockDim.x) {
      const int b0 = a.begin[i], b1 = a.begin[i + 1];
      bad |= b0 != b1 && (b0 < 0 || b1 < b0 || b1 > a.n_rows);
    }
  if (bad) kv4_flag(c, NT_KV4_BAD_LEN);
  return true;
}

// Unit u of the call: a chunk that entry i's rows may touch.  Entry i's units start
// at begin[i] / 16 + 2 i: r rows touch at most r / 16 + 2 chunks, so they do not
// meet entry i + 1's; the units between belong to nobody.  Without `begin` a unit is an
// entry.  false: nothing to do.
// All lanes call it and get the same.
__device__ __forceinline__ bool kv4_span(const Kv4& c, const Kv4Rows& a, int u, Kv4Span* sp) {
  const int lane = threadIdx.x & 31;
  int i = u, b0 = u, b1 = u + 1, start = u;
  if (a.begin) {
    int lo = 0, hi = a.n;   // entry lo .. hi - 1 has unit u (if any has)
    int step = 1;
    while (step * 32 < hi) step *= 32;
    for (; step; step /= 32) {   // 32 candidates at a time
      const int e = lo + lane * step;
      const bool before = e < hi && a.begin[e] / kKv4Chunk + 2 * e <= u;
      const uint32_t m = __ballot_sync(0xffffffffu, before);
      if (!m) return false;
      lo += (31 - __clz(m)) * step;
      hi = lo + step < hi ? lo + step : hi;
    }
    i = lo;
    b0 = a.begin[i];
    b1 = a.begin[i + 1];
    start = b0 / kKv4Chunk + 2 * i;
    if (b1 <= b0 || b0 < 0 || b1 > a.n_rows) return false;
  } else if (u >= a.n) {
    return false;
  }
  const int rows = b1 - b0;
  const int s = a.seq ? a.seq[i] : i;
  uint32_t bad = 0;
  int n = 0;
  if (s < 0 || s >= c.max_seqs) bad = NT_KV4_BAD_SEQ;
  else if ((n = c.len[s]) > c.capacity() || n < rows) bad = NT_KV4_BAD_LEN;   // (a row range above the length: no row)
  if (bad) {
    if (lane == 0 && u == start) kv4_flag(c, bad);
    return false;
  }
  if (u - start > rows / kKv4Chunk + 1) return false;   // behind the entry's last chunk (n may be 2^31 - 256: more would not fit an int)
  const int p0 = (n - rows) / kKv4Chunk * kKv4Chunk + (u - start) * kKv4Chunk;   // the chunk's first position
  if (p0 >= n) return false;
  const int first = p0 > n - rows ? p0 : n - rows;
  sp->s = s;
  sp->p0 = p0;
  sp->row = b0 + first - (n - rows);
  sp->first = first - p0;
  sp->last = n - p0 < kKv4Chunk ? n - p0 : kKv4Chunk;
  return true;
}

// The span's chunk of kv head g; NULL where there is no such page, or (append) it
// is not the sequence's own.
__device__ __forceinline__ uint8_t* kv4_span_chunk(const Kv4& c, const Kv4Rows& a, const Kv4Span& sp, int g, bool append) {
  const int page = c.table[int64_t(sp.s) * c.max_pages + sp.p0 / c.page_len];
  if (page < 0 || page >= c.n_pages || (append && c.refs[page] != 1)) {
    if ((threadIdx.x & 31) == 0) kv4_flag(c, NT_KV4_BAD_PAGE);
    return nullptr;
  }
  return c.chunk(a.layer, page, g, sp.p0 % c.page_len);
}

__device__ __forceinline__ float kv4_max_nan(float a, float b) {   // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// maxima of f16 pairs, NaN where one is
__device__ __forceinline__ uint32_t kv4_max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t kv4_abs_max2(uint32_t a, uint32_t b) { return kv4_max2(a & 0x7fff7fffu, b & 0x7fff7fffu); }
__device__ __forceinline__ float kv4_top2(uint32_t m) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
  return kv4_max_nan(f.x, f.y);
}

__device__ __forceinline__ void kv4_unpack(uint32_t w, float* x) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  x[0] = f.x; x[1] = f.y;
}

// A block of 32 source elements in registers, 16 bytes a piece.
template <class T> struct Kv4Block;
template <> struct Kv4Block<float> {
  float4 r[8];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 8; i++) r[i] = reinterpret_cast<const float4*>(p)[i];
  }
  __device__ __forceinline__ float top() const {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++)
      m = kv4_max_nan(m, kv4_max_nan(kv4_max_nan(fabsf(r[i].x), fabsf(r[i].y)), kv4_max_nan(fabsf(r[i].z), fabsf(r[i].w))));
    return m;
  }
  __device__ __forceinline__ void get(int i, float (&x)[8]) const {   // elements 8 i..
    x[0] = r[2 * i].x; x[1] = r[2 * i].y; x[2] = r[2 * i].z; x[3] = r[2 * i].w;
    x[4] = r[2 * i + 1].x; x[5] = r[2 * i + 1].y; x[6] = r[2 * i + 1].z; x[7] = r[2 * i + 1].w;
  }
};
template <> struct Kv4Block<__half> {
  uint4 r[4];
  __device__ __forceinline__ void load(const __half* p) {
#pragma unroll
    for (int i = 0; i < 4; i++) r[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ float top() const {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; i++) m = kv4_max2(m, kv4_max2(kv4_abs_max2(r[i].x, r[i].y), kv4_abs_max2(r[i].z, r[i].w)));
    return kv4_top2(m);
  }
  __device__ __forceinline__ void get(int i, float (&x)[8]) const {
    kv4_unpack(r[i].x, x); kv4_unpack(r[i].y, x + 2); kv4_unpack(r[i].z, x + 4); kv4_unpack(r[i].w, x + 6);
  }
};
template <int N> __device__ __forceinline__ void kv4_store(float* p, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; i++)
    reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
template <int N> __device__ __forceinline__ void kv4_store(__half* p, const float (&x)[N]) {
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; i++) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (N == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[N / 2 - 2], w[N / 2 - 1]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// A block's scale from its largest magnitude (NaN where one of its values is).
struct Kv4Scale {
  uint32_t bits;    // f16; 0x7e00: the block cannot be held
  float up, down;   // 1 / d a little enlarged and diminished (0 where all codes are 8)
};
__device__ __forceinline__ Kv4Scale kv4_scale(float top) {
  const float d7 = top * (1.0f / 7.0f);
  Kv4Scale s;
  s.bits = (uint32_t(__half_as_ushort(__float2half_rn(d7))) + 8u) & 0xfff0u;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(__half2float(__ushort_as_half(uint16_t(s.bits)))));
  const bool bad = s.bits > 0x6300u;   // above 896, infinite or NaN
  if (bad || s.bits == 0u) inv = 0.f;
  if (bad) s.bits = 0x7e00u;
  s.up = inv * (1.f + 0x1p-20f);
  s.down = inv * (1.f - 0x1p-20f);
  return s;
}

// Codes of 8 values, the first in the lowest bits: round(x / d) + 8, the quotient
// rounded to fp32, halves away from zero.  1 / d is known within 2^-23, so x up
// lies farther from 0 than the rounded quotient and x down nearer.
//  fp32 x: where both round to the same number, so does the quotient; `differ` gets
//    bits where they do not (a quotient within 2^-20 of a half), and the codes are
//    formed by kv4_codes_exactly.
//  f16 x (eleven bits; d has seven): x / d is a half or farther than 2^-12 of itself from
//    it, so x up rounds as the quotient does, halves away from zero.  (Halves are
//    common here: one value in a few hundred.)
// Scales below f16's normal range, whose codes may need clamping, `differ` too.
// 1.5 2^23 + 8 + q in fp32 has q + 8 in its lowest bits; the sum of the codes 16^e is
// formed modulo 2^32 with the upper bits and rid of them at the end.
template <bool F16>
__device__ __forceinline__ uint32_t kv4_codes(const float (&x)[8], const Kv4Scale& s, uint32_t& differ) {
  constexpr float kMagic = 12582920.f;
  uint32_t w = 0u;
#pragma unroll
  for (int e = 7; e >= 0; e--) {
    const uint32_t m = __float_as_uint(fmaf(x[e], s.up, kMagic));
    if (!F16) differ |= m ^ __float_as_uint(fmaf(x[e], s.down, kMagic));
    w = w * 16u + m;
  }
  return w - 0x4b400000u * 0x11111111u;
}
__device__ __noinline__ uint32_t kv4_codes_exactly(float x0, float x1, float x2, float x3, float x4, float x5, float x6,
                                                   float x7, uint32_t bits) {
  const float x[8] = {x0, x1, x2, x3, x4, x5, x6, x7}, d = __half2float(__ushort_as_half(uint16_t(bits)));
  uint32_t w = 0u;
#pragma unroll
  for (int e = 0; e < 8; e++) {
    const int q = int(roundf(__fdiv_rn(x[e], d))) + 8;
    w |= uint32_t(q < 0 ? 0 : (q > 15 ? 15 : q)) << (4 * e);
  }
  return w;
}

constexpr int kKv4RowWarps = 4;   // warps of a CTA: each K or V of a (unit, kv head)

// NG words from consecutive addresses
template <int NG>
__device__ __forceinline__ void kv4_get(const void* p, uint32_t (&w)[NG]) {
  if (NG == 4) {
    const uint4 x = *static_cast<const uint4*>(p);
    w[0] = x.x; w[1] = x.y; w[2 % NG] = x.z; w[3 % NG] = x.w;
  } else {
    const uint2 x = *static_cast<const uint2*>(p);
    w[0] = x.x; w[1] = x.y;
  }
}

template <int HD, class T>
__global__ void __launch_bounds__(32 * kKv4RowWarps) k_kv4_append(Kv4 c, Kv4Rows a, const T* k, const T* v) {
  using L = Kv4Chunk<HD>;
  constexpr int NG = L::NG, NB = NG / 2;             // blocks of a lane
  __shared__ __align__(16) uint8_t s_codes[kKv4RowWarps][8 * HD];
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t(blockIdx.x) - a.checks) * kKv4RowWarps + (threadIdx.x >> 5);   // (below 0: see kv4_check_rows)
  const int g = int(id / 2 % c.n_kv);
  const int64_t u = id / 2 / c.n_kv;
  const bool is_v = id & 1;
  if (u >= a.units) return;
  kv4_dependent();
  if (kv4_check_rows(c, a)) return;
  Kv4Span sp;
  if (!kv4_span(c, a, int(u), &sp)) return;
  const T* src = (is_v ? v : k) + int64_t(sp.row - sp.first) * a.row_stride + int64_t(g) * a.head_stride;   // of position 0
  // block 32 i + lane: position / NG, dimensions 32 (block % NG) + 0..31
  Kv4Block<T> raw[NB];
  bool live[NB];
#pragma unroll
  for (int i = 0; i < NB; i++) {
    const int b = 32 * i + lane, p = b / NG;
    live[i] = p >= sp.first && p < sp.last;
    if (live[i]) raw[i].load(src + int64_t(p) * a.row_stride + 32 * (b % NG));
  }
  uint8_t* chunk = kv4_span_chunk(c, a, sp, g, true);
  if (!chunk) return;
  uint8_t* codes = s_codes[threadIdx.x >> 5];
#pragma unroll
  for (int i = 0; i < NB; i++) {
    if (!live[i]) continue;
    const int b = 32 * i + lane, p = b / NG, j = b % NG;
    const Kv4Scale sc = kv4_scale(raw[i].top());
    *reinterpret_cast<uint16_t*>(chunk + (is_v ? L::v_scale(p, j) : L::k_scale(p, j))) = uint16_t(sc.bits);
#pragma unroll
    for (int y = 0; y < 4; y++) {
      float x[8];
      raw[i].get(y, x);
      uint32_t differ = 0u, w = kv4_codes<sizeof(T) == 2>(x, sc, differ);
      if (sc.bits - 1u < 0x3ffu) differ = 1u;
      if (sc.bits == 0x7e00u) w = 0x88888888u;
      else if (differ) w = kv4_codes_exactly(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], sc.bits);
      if (is_v) {
        *reinterpret_cast<uint16_t*>(codes + L::v_half(p, 2 * y, j) - L::kV) = uint16_t(w);
        *reinterpret_cast<uint16_t*>(codes + L::v_half(p, 2 * y + 1, j) - L::kV) = uint16_t(w >> 16);
      } else {
        *reinterpret_cast<uint32_t*>(codes + L::k_word(p, y, j)) = w;
      }
    }
  }
  __syncwarp();
  // out, 4 NG bytes a lane: of K one position's, of V two positions'
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int x = 32 * i + lane;
    const uint8_t* from = codes + x * (4 * NG);
    uint8_t* to = chunk + (is_v ? L::kV : 0) + x * (4 * NG);
    const int p = is_v ? 8 * (x >> 5) + 2 * (x & 3) : x >> 2;
    const bool live0 = p >= sp.first && p < sp.last, live1 = is_v ? p + 1 >= sp.first && p + 1 < sp.last : live0;
    if (live0 && live1) {
      if (NG == 4) *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
      else *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(from);
    } else if (live0 || live1) {   // half of each word: the other position is not of this call
#pragma unroll
      for (int j = 0; j < NG; j++) {
        const int o = 4 * j + (live0 ? 0 : 2);
        *reinterpret_cast<uint16_t*>(to + o) = *reinterpret_cast<const uint16_t*>(from + o);
      }
    }
  }
}

// N values of the codes in w's lowest bits, exactly.
template <int N>
__device__ __forceinline__ void kv4_values(uint32_t w, float d, float (&x)[N]) {
#pragma unroll
  for (int e = 0; e < N; e++) x[e] = __fmul_rn(d, float(int((w >> (4 * e)) & 15u) - 8));
}

template <int HD, class T>
__global__ void __launch_bounds__(32 * kKv4RowWarps) k_kv4_read(Kv4 c, Kv4Rows a, T* k, T* v) {
  using L = Kv4Chunk<HD>;
  constexpr int NG = L::NG;
  const int lane = threadIdx.x & 31, gi = lane >> 2, tg = lane & 3;
  const int64_t id = (int64_t(blockIdx.x) - a.checks) * kKv4RowWarps + (threadIdx.x >> 5);   // (below 0: see kv4_check_rows)
  const int g = int(id / 2 % c.n_kv);
  const int64_t u = id / 2 / c.n_kv;
  if (u >= a.units) return;
  kv4_dependent();
  if (kv4_check_rows(c, a)) return;
  Kv4Span sp;
  if (!kv4_span(c, a, int(u), &sp)) return;
  const uint8_t* chunk = kv4_span_chunk(c, a, sp, g, false);
  if (!chunk) return;
  const int64_t row0 = int64_t(sp.row - sp.first) * a.row_stride + int64_t(g) * a.head_stride;
  uint32_t w[2][NG], s[2][NG];
  if (!(id & 1)) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      kv4_get<NG>(chunk + L::k_word(8 * i + gi, tg, 0), w[i]);
      if (NG == 4) {
        const uint2 y = *reinterpret_cast<const uint2*>(chunk + L::k_scale(8 * i + gi, 0));
        s[i][0] = y.x; s[i][1] = y.y;
      } else {
        s[i][0] = *reinterpret_cast<const uint32_t*>(chunk + L::k_scale(8 * i + gi, 0));
      }
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int p = 8 * i + gi;
      if (8 * i >= sp.last || 8 * i + 8 <= sp.first) continue;
      const bool live = p >= sp.first && p < sp.last;
      T* r = k + row0 + int64_t(p) * a.row_stride;
#pragma unroll
      for (int j = 0; j < NG; j++) {
        const float d = __half2float(__ushort_as_half(uint16_t(s[i][j >> 1] >> (16 * (j & 1)))));
        if constexpr (sizeof(T) == 2) {
          float x[8];
          kv4_values<8>(w[i][j], d, x);
          if (live) kv4_store<8>(r + 32 * j + 8 * tg, x);
        } else {   // runs of 4 that lie side by side across the lanes: tg and 4 + tg
          const uint32_t y = __shfl_sync(0xffffffffu, w[i][j], (lane & ~3) | (tg >> 1));
          const uint32_t z = __shfl_sync(0xffffffffu, w[i][j], (lane & ~3) | 2 | (tg >> 1));
          float x[4];
          kv4_values<4>(y >> (16 * (tg & 1)), d, x);
          if (live) kv4_store<4>(r + 32 * j + 4 * tg, x);
          kv4_values<4>(z >> (16 * (tg & 1)), d, x);
          if (live) kv4_store<4>(r + 32 * j + 16 + 4 * tg, x);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      kv4_get<NG>(chunk + L::v_half(8 * i + 2 * tg, gi, 0), w[i]);
      kv4_get<NG>(chunk + L::v_scale(8 * i + 2 * tg, 0), s[i]);
    }
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int y = 0; y < 2; y++) {
        const int p = 8 * i + 2 * tg + y;
        if (p < sp.first || p >= sp.last) continue;
        T* r = v + row0 + int64_t(p) * a.row_stride;
#pragma unroll
        for (int j = 0; j < NG; j++) {
          const float d = __half2float(__ushort_as_half(uint16_t(s[i][j] >> (16 * y))));
          float x[4];
          kv4_values<4>(w[i][j] >> (16 * y), d, x);
          kv4_store<4>(r + 32 * j + 4 * gi, x);
        }
      }
  }
}

// Flags sequences listed twice.
__global__ void __launch_bounds__(1024) k_kv4_listed_twice(Kv4 c, int n, const int32_t* seq) {
  kv4_dependent();
  __shared__ uint32_t set[kKv4MaxSeqs / 32];
  for (int i = threadIdx.x; i < kKv4MaxSeqs / 32; i += blockDim.x) set[i] = 0u;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int s = seq[i];
    if (s < 0 || s >= c.max_seqs) continue;
    if (atomicOr(&set[s >> 5], 1u << (s & 31)) >> (s & 31) & 1u) kv4_flag(c, NT_KV4_BAD_SEQ);
  }
}

// ------------------------------------------------------------ page operators --

// Exclusive prefix sum of one value per thread of a 1024-thread CTA; *total: the sum.
__device__ __forceinline__ int64_t kv4_scan(int64_t x, int64_t* total) {
  __shared__ int64_t part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  __syncthreads();   // (the sums of the call before have been read)
  if (lane == 31) part[warp] = s;
  __syncthreads();
  int64_t w = part[lane];
  const int64_t mine = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  return __shfl_sync(0xffffffffu, w - mine, warp) + s - x;
}

__device__ __forceinline__ int kv4_pages(int len, int page_len) { return int((int64_t(len) + page_len - 1) / page_len); }

struct Kv4PlanArgs {
  int32_t n;
  const int32_t* a;   // extend: sequences (nullable); fork: sources
  const int32_t* b;   // extend: counts; fork: destinations
  const int32_t* keep;
  int32_t* go;        // [0]: the call goes ahead, [1]: pages to copy
  int64_t* off;
  int32_t* from;      // page that entry i's first new page is a copy of (-1: none)
  int2* pair;
  int32_t* free;
};

// The plan of an extend (FORK = false) or a fork, by one CTA: checks every entry and
// every page that it will share or copy, counts the pages it takes, finds that many free pages, the lowest first, and
// writes their table entries and counts, and (extend) the lengths.  Nothing is changed unless every
// entry is valid and the free pages suffice.  The pages to copy go to `pair`.
template <bool FORK>
__global__ void __launch_bounds__(1024, 1) k_kv4_plan(Kv4 c, Kv4PlanArgs a) {
  __shared__ uint32_t set[kKv4MaxSeqs / 32];                  // sequences listed (fork: destinations)
  __shared__ uint32_t s_bad;
  __shared__ int s_pairs;
  const int t = threadIdx.x;
  for (int i = t; i < kKv4MaxSeqs / 32; i += 1024) set[i] = 0u;
  if (t == 0) { s_bad = 0u; s_pairs = 0; }
  kv4_dependent();
  // (fork) 2^lg threads look at a source's full pages: all 1024 shared out to the entries, at least 8 each, the last threads first
  const int ceil_lg = 32 - __clz(a.n - 1), lg = ceil_lg < 7 ? 10 - ceil_lg : 3;
  const int i_pages = (1023 - t) >> lg, j_pages = (1023 - t) & ((1 << lg) - 1);
  // on the way while the entries are checked: counts of the first pages, and (fork) the sources that this thread begins with
  const int refs0 = t < c.n_pages ? c.refs[t] : 1;
  const int src0 = FORK && t < a.n ? a.a[t] : 0, src1 = FORK && i_pages < a.n ? a.a[i_pages] : 0;
  __syncthreads();
  const int32_t* listed = FORK ? a.b : a.a;
  for (int i = t; i < a.n; i += 1024) {
    const int s = listed ? listed[i] : i;
    if (s < 0 || s >= c.max_seqs || (atomicOr(&set[s >> 5], 1u << (s & 31)) >> (s & 31) & 1u))
      atomicOr(&s_bad, NT_KV4_BAD_SEQ);
  }
  __syncthreads();
  if (FORK) {   // the full pages to be shared
    for (int i = i_pages; i < a.n; i += 1024 >> lg) {
      const int s = i == i_pages ? src1 : a.a[i];
      if (s < 0 || s >= c.max_seqs) continue;
      const int n = c.len[s], keep = a.keep ? a.keep[i] : n, full = keep / c.page_len;
      if (n > c.capacity() || keep > n) continue;
      const int32_t* row = c.table + int64_t(s) * c.max_pages;
      bool bad = false;
#pragma unroll 4
      for (int j = j_pages; j < full; j += 1 << lg) {
        const int p = row[j];
        bad |= p < 0 || p >= c.n_pages || c.refs[p] < 1;
      }
      if (bad) atomicOr(&s_bad, NT_KV4_BAD_PAGE);
    }
  }
  int64_t run = 0;   // pages taken by the entries before
  for (int i0 = 0; i0 < a.n; i0 += 1024) {
    const int i = i0 + t;
    int64_t need = 0;
    int from = -1;
    uint32_t bad = 0;
    if (i < a.n) {
      const int s = FORK && i == t ? src0 : a.a ? a.a[i] : i;   // the sequence read from
      if (s < 0 || s >= c.max_seqs) {
        bad = NT_KV4_BAD_SEQ;
      } else {
        const int n = c.len[s], held = n < 0 || n > c.capacity() ? 0 : kv4_pages(n, c.page_len);
        if (n < 0 || n > c.capacity()) bad |= NT_KV4_BAD_LEN;
        if (FORK) {
          const int keep = a.keep ? a.keep[i] : n, d = a.b[i];
          if (set[s >> 5] >> (s & 31) & 1u) bad |= NT_KV4_BAD_SEQ;
          if (d >= 0 && d < c.max_seqs && c.len[d] != 0) bad |= NT_KV4_BAD_SEQ;
          if (keep < 0 || keep > n) bad |= NT_KV4_BAD_LEN;
          if (!bad && keep % c.page_len) {
            from = c.table[int64_t(s) * c.max_pages + keep / c.page_len];
            if (from < 0 || from >= c.n_pages || c.refs[from] < 1) bad |= NT_KV4_BAD_PAGE;
            need = 1;
          }
        } else {
          const int count = a.b[i];
          if (count < 0 || count > c.capacity() - n) bad |= NT_KV4_BAD_LEN;
          if (!bad && count > 0) {
            need = kv4_pages(n + count, c.page_len) - held;
            if (n % c.page_len) {
              const int p = c.table[int64_t(s) * c.max_pages + n / c.page_len];
              if (p < 0 || p >= c.n_pages || c.refs[p] < 1) bad |= NT_KV4_BAD_PAGE;
              else if (c.refs[p] > 1) { from = p; need++; }
            }
          }
        }
      }
      if (bad) atomicOr(&s_bad, bad);
      a.from[i] = from;
    }
    int64_t all;
    const int64_t before = kv4_scan(need, &all);
    if (i < a.n) a.off[i] = run + before;
    run += all;
  }
  if (t == 0) a.off[a.n] = run;
  // the lowest `run` free pages
  int64_t found = 0;
  for (int64_t p0 = 0; p0 < c.n_pages && found < run; p0 += 1024) {
    const int64_t p = p0 + t;
    const bool is_free = p < c.n_pages && (p0 ? c.refs[p] : refs0) == 0;
    int64_t all;
    const int64_t before = kv4_scan(is_free ? 1 : 0, &all);
    if (is_free && found + before < run) a.free[found + before] = int32_t(p);
    found += all;
  }
  __syncthreads();
  if (found < run && t == 0 && !s_bad) s_bad = NT_KV4_NO_PAGE;
  __syncthreads();
  const uint32_t bad = s_bad;
  if (t == 0) {
    a.go[0] = bad == 0u;
    if (bad) a.go[1] = 0;
    if (bad) kv4_flag(c, bad);
  }
  if (bad) return;
  for (int64_t f = t; f < run; f += 1024) {   // free page f belongs to the entry with off[lo] <= f < off[lo + 1]
    int lo = 0, hi = a.n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.off[mid] <= f) lo = mid; else hi = mid;
    }
    const int page = a.free[f], kth = int(f - a.off[lo]);
    c.refs[page] = 1;
    const bool copied = a.from[lo] >= 0;
    if (copied && kth == 0) a.pair[atomicAdd(&s_pairs, 1)] = make_int2(a.from[lo], page);   // (in any order)
    if (FORK) {
      const int keep = a.keep ? a.keep[lo] : c.len[a.a[lo]];
      c.table[int64_t(a.b[lo]) * c.max_pages + keep / c.page_len] = page;
    } else {
      const int s = a.a ? a.a[lo] : lo, n = c.len[s];
      const int slot = copied ? n / c.page_len + kth : kv4_pages(n, c.page_len) + kth;
      int32_t* e = &c.table[int64_t(s) * c.max_pages + slot];
      if (copied && kth == 0) atomicSub(&c.refs[*e], 1);
      *e = page;
    }
  }
  __syncthreads();
  if (t == 0) a.go[1] = s_pairs;
  if (!FORK)
    for (int i = t; i < a.n; i += 1024) c.len[a.a ? a.a[i] : i] += a.b[i];
}

// ---- copies.  Whole pages move in pieces through shared memory by bulk copies:
// one thread of each of a CTA's first warps has a ring of its own, kKv4Ahead pieces on
// the way in while others are on the way out; the remaining warps do what else there
// is.  (Copies by all threads, 64 bytes each in flight, 8 CTAs of 256 per SM: 53.6
// us for 24 pages of 73.7 KB in 80 layers.)
constexpr int kKv4Streams = 4, kKv4Piece = 12288, kKv4Ring = 4, kKv4Ahead = 3;
constexpr int kKv4CopyThreads = 256;
struct Kv4CopyShared {   // of a stream
  static constexpr int kBars = kKv4Piece * kKv4Ring, kTo = kBars + 8 * kKv4Ring, kBytes = kTo + 8 * kKv4Ring,
                       kStream = (kBytes + 4 * kKv4Ring + 127) / 128 * 128, kSize = kStream * kKv4Streams;
  static_assert(kSize <= 220 * 1024, "shared memory of a CTA");
};
extern __shared__ __align__(128) uint8_t kv4_sm[];

// Pieces of n pages of every layer: `count` of `bytes` each (the last of a page the rest).
struct Kv4Pieces {
  int32_t bytes, count;
};
// 12 KB, or less where that makes fewer pieces than streams (1 KB at least).
static Kv4Pieces kv4_pieces(const Kv4& k, int64_t n) {
  const int64_t pb = k.page_bytes(), all = pb * k.n_layers * n;
  int64_t b = kKv4Piece;
  while (b > 1024 && all / b < kKv4Streams * 152) b /= 2;
  Kv4Pieces p;
  p.count = int32_t((pb + b - 1) / b);
  p.bytes = int32_t(((pb + p.count - 1) / p.count + 15) / 16 * 16);
  p.count = int32_t((pb + p.bytes - 1) / p.bytes);
  return p;
}

// The stream's share of the pieces of `pairs` pages (source, destination) in every
// layer, one after the other; by the calling thread.  pair(i): the i-th pair (x < 0:
// it is not copied).  No pair's destination is another's source.
template <class P>
__device__ __forceinline__ void kv4_stream(const Kv4& c, Kv4Pieces ps, int64_t pairs, int stream, P pair) {
  using Sh = Kv4CopyShared;
  const int64_t per = int64_t(c.n_layers) * ps.count, all = pairs * per, streams = int64_t(gridDim.x) * kKv4Streams;
  const int64_t each = (all + streams - 1) / streams, q0 = (int64_t(blockIdx.x) * kKv4Streams + stream) * each;
  int64_t todo = q0 + each < all ? each : all - q0;   // pieces not yet begun
  if (todo <= 0) return;
  uint8_t* sm = kv4_sm + stream * Sh::kStream;
  const uint32_t ring = kv4_smem(sm), bars = ring + Sh::kBars;
  uint8_t** to = reinterpret_cast<uint8_t**>(sm + Sh::kTo);
  uint32_t* bytes = reinterpret_cast<uint32_t*>(sm + Sh::kBytes);
  for (int i = 0; i < kKv4Ring; i++) kv4_bar_init(bars + 8 * i);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  const int64_t pb = c.page_bytes();
  int64_t i = q0 / per;
  int layer = int(q0 % per / ps.count), part = int(q0 % ps.count);
  int2 m = pair(i);
  uint32_t in = 0, out = 0;   // pieces whose copy in, out was begun
  for (;;) {
    while (todo > 0 && in - out < kKv4Ahead) {
      if (m.x >= 0) {
        const int st = in % kKv4Ring;
        // the copy out of what stood there before has been read: all but the last kKv4Ring - kKv4Ahead have
        asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kKv4Ring - kKv4Ahead) : "memory");
        const int64_t at = int64_t(part) * ps.bytes, plane = int64_t(layer) * c.n_pages;
        const uint32_t n = uint32_t(pb - at < ps.bytes ? pb - at : ps.bytes);
        to[st] = c.pool + (plane + m.y) * pb + at;
        bytes[st] = n;
        kv4_bar_expect(bars + 8 * st, n);
        kv4_copy(ring + st * kKv4Piece, c.pool + (plane + m.x) * pb + at, n, bars + 8 * st);
        in++;
      }
      todo--;
      if (++part == ps.count) {
        part = 0;
        if (++layer == c.n_layers) {
          layer = 0;
          i++;
          if (todo > 0) m = pair(i);
        }
      }
    }
    if (out == in) break;
    const int st = out % kKv4Ring;
    if (!kv4_bar_wait(bars + 8 * st, out / kKv4Ring & 1u)) {
      kv4_flag(c, NT_KV4_TIMEOUT);
      for (uint32_t x = out + 1; x < in; x++) kv4_bar_wait(bars + 8 * (x % kKv4Ring), x / kKv4Ring & 1u);
      break;
    }
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;" ::"l"(to[st]),
                 "r"(ring + st * kKv4Piece), "r"(bytes[st])
                 : "memory");
    out++;
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// The pairs of a plan; FORK: also the destinations' tables, counts and lengths.
template <bool FORK>
__global__ void __launch_bounds__(kKv4CopyThreads) k_kv4_apply(Kv4 c, Kv4PlanArgs a, Kv4Pieces ps) {
  kv4_dependent();
  if (!a.go[0]) return;
  const int warp = threadIdx.x >> 5;
  if (warp < kKv4Streams) {
    if ((threadIdx.x & 31) == 0) kv4_stream(c, ps, a.go[1], warp, [&](int64_t i) { return a.pair[i]; });
    return;
  }
  if (FORK) {
    constexpr int kFirst = 32 * kKv4Streams;
    for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
      const int s = a.a[i], d = a.b[i], keep = a.keep ? a.keep[i] : c.len[s], full = keep / c.page_len;
      const int32_t* from = c.table + int64_t(s) * c.max_pages;
      int32_t* to = c.table + int64_t(d) * c.max_pages;
      for (int j = threadIdx.x - kFirst; j < full; j += kKv4CopyThreads - kFirst) {
        const int p = from[j];   // (the plan has checked it)
        to[j] = p;
        atomicAdd(&c.refs[p], 1);
      }
      if (threadIdx.x == kFirst) c.len[d] = keep;
    }
  }
}

__global__ void __launch_bounds__(256) k_kv4_free(Kv4 c, int n, const int32_t* seq, const int32_t* keep) {
  __shared__ int s_again;
  kv4_dependent();
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int s = seq ? seq[i] : i;
    __syncthreads();
    if (threadIdx.x == 0) s_again = 0;
    __syncthreads();
    if (seq)
      for (int e = threadIdx.x; e < i; e += blockDim.x)
        if (seq[e] == s) s_again = 1;
    __syncthreads();
    if (s < 0 || s >= c.max_seqs || s_again) {
      if (threadIdx.x == 0) kv4_flag(c, NT_KV4_BAD_SEQ);
      continue;
    }
    const int len = c.len[s], left = keep ? keep[i] : 0;
    if (len < 0 || len > c.capacity() || left < 0 || left > len) {
      if (threadIdx.x == 0) kv4_flag(c, NT_KV4_BAD_LEN);
      continue;
    }
    int32_t* row = c.table + int64_t(s) * c.max_pages;
    for (int j = kv4_pages(left, c.page_len) + int(threadIdx.x); j < kv4_pages(len, c.page_len); j += blockDim.x) {
      const int p = row[j];
      row[j] = -1;
      if (p < 0 || p >= c.n_pages) { kv4_flag(c, NT_KV4_BAD_PAGE); continue; }
      if (atomicSub(&c.refs[p], 1) < 1) {   // nobody held it
        atomicAdd(&c.refs[p], 1);
        kv4_flag(c, NT_KV4_BAD_PAGE);
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) c.len[s] = left;
  }
}

// A CTA's pieces belong to few pairs: those are checked first.
constexpr int kKv4CopyPairs = 8192;   // most pairs of a CTA: 2^20 pairs over at least 130
__global__ void __launch_bounds__(kKv4CopyThreads) k_kv4_copy_pages(Kv4 c, int n, const int32_t* src, const int32_t* dst,
                                                                    Kv4Pieces ps) {
  __shared__ uint32_t s_bad[kKv4CopyPairs / 32];
  kv4_dependent();
  const int64_t per = int64_t(c.n_layers) * ps.count, all = n * per, streams = int64_t(gridDim.x) * kKv4Streams;
  const int64_t each = (all + streams - 1) / streams * kKv4Streams, q0 = blockIdx.x * each, q1 = q0 + each < all ? q0 + each : all;
  if (q0 >= q1) return;
  const int i0 = int(q0 / per), i1 = int((q1 - 1) / per);
  for (int i = threadIdx.x; i <= (i1 - i0) / 32; i += kKv4CopyThreads) s_bad[i] = 0u;
  __syncthreads();
  for (int i = i0; i <= i1; i++) {
    const int s = src[i], d = dst[i];
    bool bad = s < 0 || s >= c.n_pages || d < 0 || d >= c.n_pages;
    for (int e = threadIdx.x; e < n; e += kKv4CopyThreads) {
      const int x = dst[e];
      bad = bad || (e != i && (x == s || (e < i && x == d)));
    }
    if (bad) {
      atomicOr(&s_bad[(i - i0) >> 5], 1u << ((i - i0) & 31));
      kv4_flag(c, NT_KV4_BAD_PAGE);
    }
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  if (warp < kKv4Streams && (threadIdx.x & 31) == 0)
    kv4_stream(c, ps, n, warp, [&](int64_t q) {
      const int i = int(q), s = src[i], d = dst[i];
      return (s_bad[(i - i0) >> 5] >> ((i - i0) & 31) & 1u) || s == d ? make_int2(-1, -1) : make_int2(s, d);
    });
}

// The plan of a compaction by one CTA: L, the pages in use; `to[p]`, where page p
// goes (or -2 for a free page below L, which receives another, -3 for one from L on); the moves
// in `pair`, the k-th page in use from L on to the k-th free page below.
__global__ void __launch_bounds__(1024) k_kv4_compact_plan(Kv4 c, int32_t* go, int2* pair, int32_t* to, int32_t* live) {
  const int t = threadIdx.x;
  kv4_dependent();
  int64_t used = 0;
  for (int64_t p0 = 0; p0 < c.n_pages; p0 += 1024) {
    int64_t all;
    kv4_scan(p0 + t < c.n_pages && c.refs[p0 + t] > 0 ? 1 : 0, &all);
    used += all;
  }
  int64_t holes = 0, movers = 0;
  for (int64_t p0 = 0; p0 < c.n_pages; p0 += 1024) {
    const int64_t p = p0 + t;
    const bool in = p < c.n_pages, use = in && c.refs[p] > 0;
    const bool hole = in && !use && p < used, mover = use && p >= used;
    int64_t nh, nm;
    const int64_t h = holes + kv4_scan(hole ? 1 : 0, &nh), m = movers + kv4_scan(mover ? 1 : 0, &nm);
    if (hole) pair[h].y = int32_t(p);
    if (mover) pair[m].x = int32_t(p);
    if (in) to[p] = hole ? -2 : (use ? int32_t(p) : -3);
    holes += nh;
    movers += nm;
  }
  __syncthreads();
  for (int64_t i = t; i < movers; i += 1024) to[pair[i].x] = pair[i].y;
  if (t == 0) {
    go[1] = int32_t(movers);
    *live = int32_t(used);
  }
}

__global__ void __launch_bounds__(kKv4CopyThreads) k_kv4_compact_apply(Kv4 c, const int32_t* go, const int2* pair, const int32_t* to,
                                                           int32_t* table_out, int32_t* refs_out, Kv4Pieces ps) {
  kv4_dependent();
  const int warp = threadIdx.x >> 5;
  if (warp < kKv4Streams) {
    if ((threadIdx.x & 31) == 0) kv4_stream(c, ps, go[1], warp, [&](int64_t i) { return pair[i]; });
    return;
  }
  constexpr int kOthers = kKv4CopyThreads - 32 * kKv4Streams;   // the other warps write tables and counts
  const int64_t first = int64_t(blockIdx.x) * kOthers + threadIdx.x - 32 * kKv4Streams, step = int64_t(gridDim.x) * kOthers;
  for (int64_t p = first; p < c.n_pages; p += step) {
    const int d = to[p], r = c.refs[p];
    if (d == -2) continue;                     // the page that moves here writes it
    if (d >= 0 && d != int(p)) refs_out[d] = r;
    refs_out[p] = d < 0 || d == int(p) ? r : 0;
  }
  for (int64_t e = first; e < int64_t(c.max_seqs) * c.max_pages; e += step) {
    int p = c.table[e];
    bool bad = p < -1 || p >= c.n_pages;
    if (p >= 0 && !bad) {
      p = to[p];
      bad = p < 0;               // it names a free page: it holds nothing
      if (bad) p = -1;
    }
    if (bad) kv4_flag(c, NT_KV4_BAD_PAGE);
    table_out[e] = p;
  }
}

// A copying kernel: one CTA per SM, fewer where there are fewer pieces.
template <class K, class... A>
static cudaError_t kv4_launch_copy(const KernelSetup& setup, K kern, int64_t pieces, cudaStream_t s, A... args) {
  if (setup.err != cudaSuccess) return setup.err;
  const int64_t ctas = (pieces + kKv4Streams - 1) / kKv4Streams;
  const unsigned grid = unsigned(ctas < 1 ? 1 : (ctas < setup.sms ? ctas : setup.sms));
  return kv4_launch_smem(kern, grid, kKv4CopyThreads, Kv4CopyShared::kSize, s, args...);
}

static unsigned kv4_grid(int64_t blocks, int64_t most) { return unsigned(blocks < 1 ? 1 : (blocks > most ? most : blocks)); }

static nt_status kv4_ws_check(const Kv4& k, const char* who, int64_t n, void* ws, size_t bytes, Kv4Ws* w) {
  *w = kv4_ws(k, n);
  if (!kv4_aligned(ws, 16)) return fail(NT_E_INVAL, std::string(who) + ": workspace is NULL or not 16-byte aligned");
  if (bytes < w->bytes) return fail(NT_E_INVAL, std::string(who) + ": workspace too small");
  if (kv4_meets_cache(k, ws, int64_t(w->bytes))) return fail(NT_E_INVAL, std::string(who) + ": the workspace overlaps the cache");
  return NT_OK;
}

static nt_status kv4_list_check(const Kv4& k, const char* who, int64_t n, int64_t most) {
  if (n < 0 || n > most) return fail(NT_E_INVAL, std::string(who) + ": more entries than the cache has, or fewer than 0");
  return NT_OK;
}

// A list of n int32 on the device: aligned, and apart from the cache and the workspace.
static nt_status kv4_array_check(const Kv4& k, const char* who, const void* p, int64_t n, bool nullable, const void* ws,
                                 size_t ws_bytes) {
  if (!p && nullable) return NT_OK;
  if (!kv4_aligned(p, 4)) return fail(NT_E_INVAL, std::string(who) + ": a list is NULL or not 4-byte aligned");
  if (kv4_meets_cache(k, p, n * 4) || (ws && kv4_overlap(p, n * 4, ws, int64_t(ws_bytes))))
    return fail(NT_E_INVAL, std::string(who) + ": a list overlaps the cache or the workspace");
  return NT_OK;
}

template <bool FORK>
static nt_status kv4_plan_apply(const char* who, const Kv4& k, Kv4PlanArgs a, void* ws, size_t ws_bytes, void* stream) {
  Kv4Ws w;
  nt_status st = kv4_ws_check(k, who, a.n, ws, ws_bytes, &w);
  if (!st) st = kv4_array_check(k, who, a.a, a.n, !FORK, ws, w.bytes);
  if (!st) st = kv4_array_check(k, who, a.b, a.n, false, ws, w.bytes);
  if (!st) st = kv4_array_check(k, who, a.keep, a.n, true, ws, w.bytes);
  if (st || a.n == 0) return st;
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.go = reinterpret_cast<int32_t*>(base);
  a.off = reinterpret_cast<int64_t*>(base + w.off);
  a.from = reinterpret_cast<int32_t*>(base + w.from);
  a.pair = reinterpret_cast<int2*>(base + w.pair);
  a.free = reinterpret_cast<int32_t*>(base + w.free);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  NT_CUDA(kv4_launch(k_kv4_plan<FORK>, 1u, 1024u, s, k, a));
  static const KernelSetup setup = kernel_setup(k_kv4_apply<FORK>, Kv4CopyShared::kSize);
  const Kv4Pieces ps = kv4_pieces(k, a.n);
  NT_CUDA(kv4_launch_copy(setup, k_kv4_apply<FORK>, int64_t(a.n) * k.n_layers * ps.count, s, k, a, ps));
  return NT_OK;
}

// Units of a call (see kv4_span), at most 2^26, so that begin / 16 + 2 i and the grid
// fit 31 bits (0: n or n_rows is out of range).
static int32_t kv4_units(int32_t n, int32_t n_rows, const int32_t* begin) {
  const int64_t u = begin ? int64_t(n_rows) / kKv4Chunk + 2 * int64_t(n) + 1 : (n < n_rows ? n : n_rows);
  return n < 0 || n_rows < 0 || u > (1 << 26) ? 0 : int32_t(u);
}

// CTAs that look over the entries.
static int32_t kv4_checks(int32_t n, int32_t n_rows, const int32_t* begin) {
  return begin ? int32_t((int64_t(n) + kKv4CheckEntries - 1) / kKv4CheckEntries) : n > n_rows;
}

static nt_status kv4_rows_check(const char* who, const Kv4& k, const Kv4Rows& a, nt_qtype type, const void* pk, const void* pv) {
  auto bad = [&](const char* what) { return fail(NT_E_INVAL, std::string(who) + ": " + what); };
  if (type != NT_F32 && type != NT_F16) return bad("type must be NT_F32 or NT_F16");
  if (a.layer < 0 || a.layer >= k.n_layers) return bad("layer out of range");
  if (a.n < 0 || (!a.seq && a.n > k.max_seqs)) return bad("n out of range");
  if (a.n_rows < 0) return bad("n_rows must not be negative");
  if (a.n && a.n_rows && !a.units) return bad("n_rows / 16 + 2 n above 2^26");
  if (int64_t(a.units) * k.n_kv > (int64_t(1) << 32) - (1 << 17))   // (so that a.units n_kv / 2 + a.checks CTAs are a grid)
    return bad("n_kv_heads (n_rows / 16 + 2 n) above 2^32 - 2^17");
  const int64_t es = type == NT_F32 ? 4 : 2, most = int64_t(1) << 40;
  if (a.row_stride < 0 || a.head_stride < 0 || a.row_stride > most || a.head_stride > most || a.row_stride * es % 16 ||
      a.head_stride * es % 16)
    return bad("strides must be multiples of 16 bytes and not negative");
  if (!kv4_aligned(pk, 16) || !kv4_aligned(pv, 16)) return bad("k or v is NULL or not 16-byte aligned");
  return NT_OK;
}

// Bytes from the first to the last element of the rows (-1: beyond 2^60).
static int64_t kv4_rows_bytes(const Kv4& k, const Kv4Rows& a, nt_qtype type) {
  const double most = double(a.n_rows) * double(a.row_stride) + double(k.n_kv) * double(a.head_stride);
  if (most > 1e17) return -1;
  return ((int64_t(a.n_rows) - 1) * a.row_stride + int64_t(k.n_kv - 1) * a.head_stride + k.hd) * (type == NT_F32 ? 4 : 2);
}

// Whether a (row, kv head) vector of one tensor shares bytes with one of another
// of the same strides that starts d bytes further (same: the tensor itself, each
// vector apart from itself).
static bool kv4_rows_meet(const Kv4& k, const Kv4Rows& a, int64_t es, int64_t d, bool same) {
  const int64_t rs = a.row_stride * es, hs = a.head_stride * es, w = k.hd * es;
  for (int64_t h = -(k.n_kv - 1); h <= k.n_kv - 1; h++) {
    const int64_t x = d + h * hs;                 // then + r rs, r in (-n_rows, n_rows)
    int64_t r0 = rs ? -x / rs : 0;                // near the row difference that brings it to 0, or the nearest there is
    r0 = r0 < 1 - int64_t(a.n_rows) ? 1 - int64_t(a.n_rows) : (r0 > int64_t(a.n_rows) - 1 ? int64_t(a.n_rows) - 1 : r0);
    for (int64_t r = r0 - 1; r <= r0 + 1; r++) {
      if (r <= -int64_t(a.n_rows) || r >= a.n_rows || (same && r == 0 && h == 0)) continue;
      const int64_t y = x + r * rs;
      if (y > -w && y < w) return true;
    }
  }
  return false;
}

}  // namespace nt

using namespace nt;

extern "C" {

nt_status nt_kv4_pool_bytes(const nt_kv4_cache* c, size_t* page_bytes, size_t* pool_bytes) {
  Kv4 k;
  const nt_status st = kv4_check(c, "nt_kv4_pool_bytes", false, &k);
  if (st) return st;
  if (page_bytes) *page_bytes = size_t(k.page_bytes());
  if (pool_bytes) *pool_bytes = size_t(k.page_bytes()) * size_t(k.n_pages) * size_t(k.n_layers);
  return NT_OK;
}

nt_status nt_kv4_workspace_bytes(const nt_kv4_cache* c, int32_t n_heads, int32_t n, size_t* bytes) {
  Kv4 k;
  const nt_status st = kv4_check(c, "nt_kv4_workspace_bytes", false, &k);
  if (st) return st;
  if (!bytes) return fail(NT_E_INVAL, "nt_kv4_workspace_bytes: NULL argument");
  if (n < 0 || n_heads < 1) return fail(NT_E_INVAL, "nt_kv4_workspace_bytes: n or n_heads out of range");
  if (n_heads % k.n_kv) return fail(NT_E_INVAL, "nt_kv4_workspace_bytes: n_heads must be a multiple of n_kv_heads");
  const size_t a = kv4_ws(k, n).bytes, b = kv4_attn_ws_bytes(n_heads, k.n_kv, k.hd);
  *bytes = a > b ? a : b;
  return NT_OK;
}

nt_status nt_kv4_extend(const nt_kv4_cache* c, int32_t n, const int32_t* dev_seq, const int32_t* dev_count,
                        void* dev_workspace, size_t workspace_bytes, void* stream) {
  Kv4 k;
  nt_status st = kv4_check(c, "nt_kv4_extend", true, &k);
  if (!st) st = kv4_list_check(k, "nt_kv4_extend", n, k.max_seqs);
  if (st) return st;
  Kv4PlanArgs a{};
  a.n = n;
  a.a = dev_seq;
  a.b = dev_count;
  return kv4_plan_apply<false>("nt_kv4_extend", k, a, dev_workspace, workspace_bytes, stream);
}

nt_status nt_kv4_fork(const nt_kv4_cache* c, int32_t n, const int32_t* dev_src, const int32_t* dev_dst,
                      const int32_t* dev_keep, void* dev_workspace, size_t workspace_bytes, void* stream) {
  Kv4 k;
  nt_status st = kv4_check(c, "nt_kv4_fork", true, &k);
  if (!st) st = kv4_list_check(k, "nt_kv4_fork", n, k.max_seqs);
  if (st) return st;
  Kv4PlanArgs a{};
  a.n = n;
  a.a = dev_src;
  a.b = dev_dst;
  a.keep = dev_keep;
  return kv4_plan_apply<true>("nt_kv4_fork", k, a, dev_workspace, workspace_bytes, stream);
}

nt_status nt_kv4_free(const nt_kv4_cache* c, int32_t n, const int32_t* dev_seq, const int32_t* dev_keep, void* stream) {
  Kv4 k;
  nt_status st = kv4_check(c, "nt_kv4_free", true, &k);
  if (!st) st = kv4_list_check(k, "nt_kv4_free", n, k.max_seqs);
  if (!st) st = kv4_array_check(k, "nt_kv4_free", dev_seq, n, true, nullptr, 0);
  if (!st) st = kv4_array_check(k, "nt_kv4_free", dev_keep, n, true, nullptr, 0);
  if (st || n == 0) return st;
  NT_CUDA(kv4_launch(k_kv4_free, kv4_grid(n, 152 * 8), 256u, static_cast<cudaStream_t>(stream), k, n, dev_seq, dev_keep));
  return NT_OK;
}

nt_status nt_kv4_copy_pages(const nt_kv4_cache* c, int32_t n, const int32_t* dev_src, const int32_t* dev_dst,
                            void* stream) {
  Kv4 k;
  nt_status st = kv4_check(c, "nt_kv4_copy_pages", true, &k);
  if (!st) st = kv4_list_check(k, "nt_kv4_copy_pages", n, k.n_pages < (1 << 20) ? k.n_pages : 1 << 20);
  if (!st) st = kv4_array_check(k, "nt_kv4_copy_pages", dev_src, n, false, nullptr, 0);
  if (!st) st = kv4_array_check(k, "nt_kv4_copy_pages", dev_dst, n, false, nullptr, 0);
  if (st || n == 0) return st;
  static const KernelSetup setup = kernel_setup(k_kv4_copy_pages, Kv4CopyShared::kSize);
  if (setup.err == cudaSuccess && (int64_t(n) + setup.sms - 1) / setup.sms + 2 > kKv4CopyPairs)
    return fail(NT_E_UNSUPPORTED, "nt_kv4_copy_pages: too many pairs for this GPU");
  const Kv4Pieces ps = kv4_pieces(k, n);
  const int64_t pieces = int64_t(n) * k.n_layers * ps.count;
  NT_CUDA(kv4_launch_copy(setup, k_kv4_copy_pages, pieces, static_cast<cudaStream_t>(stream), k, n, dev_src, dev_dst, ps));
  return NT_OK;
}

nt_status nt_kv4_compact(const nt_kv4_cache* c, int32_t* dev_table_out, int32_t* dev_refs_out, int32_t* dev_live,
                         void* dev_workspace, size_t workspace_bytes, void* stream) {
  const char* who = "nt_kv4_compact";
  Kv4 k;
  Kv4Ws w;
  nt_status st = kv4_check(c, who, true, &k);
  if (!st) st = kv4_ws_check(k, who, 0, dev_workspace, workspace_bytes, &w);
  if (st) return st;
  const int64_t tb = int64_t(k.max_seqs) * k.max_pages * 4, rb = int64_t(k.n_pages) * 4;
  if (!kv4_aligned(dev_table_out, 4) || !kv4_aligned(dev_refs_out, 4) || !kv4_aligned(dev_live, 4))
    return fail(NT_E_INVAL, "nt_kv4_compact: an output is NULL or not 4-byte aligned");
  if ((dev_table_out != k.table && kv4_meets_cache(k, dev_table_out, tb)) ||
      (dev_refs_out != k.refs && kv4_meets_cache(k, dev_refs_out, rb)) || kv4_meets_cache(k, dev_live, 4) ||
      kv4_overlap(dev_table_out, tb, dev_refs_out, rb) || kv4_overlap(dev_table_out, tb, dev_live, 4) ||
      kv4_overlap(dev_refs_out, rb, dev_live, 4) || kv4_overlap(dev_workspace, int64_t(w.bytes), dev_table_out, tb) ||
      kv4_overlap(dev_workspace, int64_t(w.bytes), dev_refs_out, rb) ||
      kv4_overlap(dev_workspace, int64_t(w.bytes), dev_live, 4))
    return fail(NT_E_INVAL, "nt_kv4_compact: an output overlaps another buffer");
  uint8_t* base = static_cast<uint8_t*>(dev_workspace);
  int32_t* go = reinterpret_cast<int32_t*>(base);
  int2* pair = reinterpret_cast<int2*>(base + w.pair);
  int32_t* to = reinterpret_cast<int32_t*>(base + w.free);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  NT_CUDA(kv4_launch(k_kv4_compact_plan, 1u, 1024u, s, k, go, pair, to, dev_live));
  // (how many pages move is known on the device only; at most half of them do)
  static const KernelSetup setup = kernel_setup(k_kv4_compact_apply, Kv4CopyShared::kSize);
  const Kv4Pieces ps = kv4_pieces(k, k.n_pages > 16 ? k.n_pages / 8 : 1);
  NT_CUDA(kv4_launch_copy(setup, k_kv4_compact_apply, int64_t(k.n_pages) * k.n_layers * ps.count, s, k,
                          static_cast<const int32_t*>(go), static_cast<const int2*>(pair), static_cast<const int32_t*>(to),
                          dev_table_out, dev_refs_out, ps));
  return NT_OK;
}

nt_status nt_kv4_append(const nt_kv4_cache* c, int32_t layer, int32_t n, const int32_t* dev_seq,
                        const int32_t* dev_begin, int32_t n_rows, nt_qtype type, const void* dev_k, const void* dev_v,
                        int64_t row_stride, int64_t head_stride, void* stream) {
  const char* who = "nt_kv4_append";
  Kv4 k;
  nt_status st = kv4_check(c, who, true, &k);
  const Kv4Rows a{layer, n, n_rows, kv4_units(n, n_rows, dev_begin), kv4_checks(n, n_rows, dev_begin), dev_seq, dev_begin, row_stride, head_stride};
  if (!st) st = kv4_rows_check(who, k, a, type, dev_k, dev_v);
  if (!st && n > k.max_seqs) st = fail(NT_E_INVAL, "nt_kv4_append: n above max_seqs");
  if (!st) st = kv4_array_check(k, who, dev_seq, n, true, nullptr, 0);
  if (!st) st = kv4_array_check(k, who, dev_begin, int64_t(n) + 1, true, nullptr, 0);
  if (st || n == 0 || n_rows == 0) return st;
  const int64_t bytes = kv4_rows_bytes(k, a, type);
  if (bytes < 0) return fail(NT_E_INVAL, "nt_kv4_append: the strides are too large");
  if (kv4_meets_cache(k, dev_k, bytes) || kv4_meets_cache(k, dev_v, bytes))
    return fail(NT_E_INVAL, "nt_kv4_append: k or v overlaps the cache");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = unsigned((int64_t(a.units) * k.n_kv * 2 + kKv4RowWarps - 1) / kKv4RowWarps + a.checks);
  if (type == NT_F32) {
    const float *pk = static_cast<const float*>(dev_k), *pv = static_cast<const float*>(dev_v);
    NT_CUDA(k.hd == 64 ? kv4_launch(k_kv4_append<64, float>, grid, 32u * kKv4RowWarps, s, k, a, pk, pv) : kv4_launch(k_kv4_append<128, float>, grid, 32u * kKv4RowWarps, s, k, a, pk, pv));
  } else {
    const __half *pk = static_cast<const __half*>(dev_k), *pv = static_cast<const __half*>(dev_v);
    NT_CUDA(k.hd == 64 ? kv4_launch(k_kv4_append<64, __half>, grid, 32u * kKv4RowWarps, s, k, a, pk, pv) : kv4_launch(k_kv4_append<128, __half>, grid, 32u * kKv4RowWarps, s, k, a, pk, pv));
  }
  if (dev_seq && n > 1) {
    NT_CUDA(kv4_launch(k_kv4_listed_twice, 1u, 1024u, s, k, n, dev_seq));
  }
  return NT_OK;
}

nt_status nt_kv4_read(const nt_kv4_cache* c, int32_t layer, int32_t n, const int32_t* dev_seq, const int32_t* dev_begin,
                      int32_t n_rows, nt_qtype type, void* dev_k, void* dev_v, int64_t row_stride, int64_t head_stride,
                      void* stream) {
  const char* who = "nt_kv4_read";
  Kv4 k;
  nt_status st = kv4_check(c, who, true, &k);
  const Kv4Rows a{layer, n, n_rows, kv4_units(n, n_rows, dev_begin), kv4_checks(n, n_rows, dev_begin), dev_seq, dev_begin, row_stride, head_stride};
  if (!st) st = kv4_rows_check(who, k, a, type, dev_k, dev_v);
  if (!st) st = kv4_array_check(k, who, dev_seq, n, true, nullptr, 0);
  if (!st) st = kv4_array_check(k, who, dev_begin, int64_t(n) + 1, true, nullptr, 0);
  if (st || n == 0 || n_rows == 0) return st;
  const int64_t bytes = kv4_rows_bytes(k, a, type), es = type == NT_F32 ? 4 : 2;
  if (bytes < 0) return fail(NT_E_INVAL, "nt_kv4_read: the strides are too large");
  const int64_t apart = static_cast<char*>(dev_v) - static_cast<char*>(dev_k);
  if (kv4_rows_meet(k, a, es, 0, true) || (kv4_overlap(dev_k, bytes, dev_v, bytes) && kv4_rows_meet(k, a, es, apart, false)))
    return fail(NT_E_INVAL, "nt_kv4_read: rows of the outputs overlap");
  if (kv4_meets_cache(k, dev_k, bytes) || kv4_meets_cache(k, dev_v, bytes) ||
      kv4_overlap(dev_seq, int64_t(n) * 4, dev_k, bytes) || kv4_overlap(dev_seq, int64_t(n) * 4, dev_v, bytes) ||
      kv4_overlap(dev_begin, int64_t(n) * 4 + 4, dev_k, bytes) || kv4_overlap(dev_begin, int64_t(n) * 4 + 4, dev_v, bytes))
    return fail(NT_E_INVAL, "nt_kv4_read: an output overlaps another buffer");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = unsigned((int64_t(a.units) * k.n_kv * 2 + kKv4RowWarps - 1) / kKv4RowWarps + a.checks);
  if (type == NT_F32) {
    float *pk = static_cast<float*>(dev_k), *pv = static_cast<float*>(dev_v);
    NT_CUDA(k.hd == 64 ? kv4_launch(k_kv4_read<64, float>, grid, 32u * kKv4RowWarps, s, k, a, pk, pv) : kv4_launch(k_kv4_read<128, float>, grid, 32u * kKv4RowWarps, s, k, a, pk, pv));
  } else {
    __half *pk = static_cast<__half*>(dev_k), *pv = static_cast<__half*>(dev_v);
    NT_CUDA(k.hd == 64 ? kv4_launch(k_kv4_read<64, __half>, grid, 32u * kKv4RowWarps, s, k, a, pk, pv) : kv4_launch(k_kv4_read<128, __half>, grid, 32u * kKv4RowWarps, s, k, a, pk, pv));
  }
  return NT_OK;
}

}  // extern "C"
