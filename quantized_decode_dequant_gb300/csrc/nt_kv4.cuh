// nt_kv4.cuh -- layout, argument checks and workspace of the paged 4-bit K/V
// cache (include/nt.h, nt_kv4_cache), shared by its operators (nt_kv4.cu) and
// the attention over it (nt_kv4_attn.cu); and what the 8-bit cache (nt_kv8.cuh),
// whose pages differ in size and contents only, has in common with it.
#pragma once

#include "nt_internal.cuh"

namespace nt {

constexpr int kKv4Chunk = 16;          // positions of a chunk
constexpr int kKv4MaxSeqs = 65536;     // bits of the shared-memory sets of listed sequences (8 KB each)

// Bytes of one chunk of hd dimensions: 8 hd of codes and hd of scales (16 hd / 32 f16) for K and for V.
__host__ __device__ constexpr int kv4_chunk_bytes(int hd) { return 18 * hd; }

// The cache as kernels see it.
struct Kv4 {
  int32_t n_layers, n_kv, hd, page_len, n_pages, max_seqs, max_pages;
  uint8_t* pool;
  int32_t* table;
  int32_t* len;
  int32_t* refs;
  uint32_t* error;
  int64_t pb;          // bytes of a page of one layer

  __host__ __device__ int64_t page_bytes() const { return pb; }
  // chunk holding position `at` (within its page) of kv head g
  __device__ uint8_t* chunk(int layer, int page, int g, int at) const {
    return pool + (int64_t(layer) * n_pages + page) * page_bytes() +
           (int64_t(g) * (page_len / kKv4Chunk) + at / kKv4Chunk) * kv4_chunk_bytes(hd);
  }
  __device__ int capacity() const { return max_pages * page_len; }
};

// Offsets inside a chunk (p: position within it, j: 32-dimension group).
template <int HD>
struct Kv4Chunk {
  static constexpr int NG = HD / 32;
  static constexpr int kV = 8 * HD, kKS = 16 * HD, kVS = 17 * HD, kBytes = 18 * HD;
  // word of dimensions 32 j + 8 tg + 0..7 of K
  static __host__ __device__ constexpr int k_word(int p, int tg, int j) { return ((p * 4 + tg) * NG + j) * 4; }
  // half word of dimensions 32 j + 4 gi + 0..3 of V
  static __host__ __device__ constexpr int v_half(int p, int gi, int j) {
    return kV + ((((p >> 3) * 8 + gi) * 4 + ((p >> 1) & 3)) * NG + j) * 4 + (p & 1) * 2;
  }
  static __host__ __device__ constexpr int k_scale(int p, int j) { return kKS + (p * NG + j) * 2; }
  static __host__ __device__ constexpr int v_scale(int p, int j) { return kVS + (((p >> 1) * NG + j) * 2 + (p & 1)) * 2; }
};

// ------------------------------------------------------------ host checks --

inline bool kv4_aligned(const void* p, uintptr_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool kv4_overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + uintptr_t(nb) && y < x + uintptr_t(na);
}

// Checks the sizes of a description (pointers too with `pointers`) and fills k.
nt_status kv4_check(const nt_kv4_cache* c, const char* who, bool pointers, Kv4* k);
// The same for pages of page_bytes, whose page_len is right.
nt_status kv4_check_pages(const Kv4& c, const char* who, bool pointers);
// Whether [p, p + bytes) meets one of the cache's buffers.
bool kv4_meets_cache(const Kv4& k, const void* p, int64_t bytes);

// Workspace of the page operators, 16-byte aligned parts.
//   plan: int32 [4]: {the call goes ahead, pairs to copy, -, -}
//   off:  int64 [n + 1] first free page of each entry's share
//   from: int32 [n] page that an entry's first new page is a copy of (-1: none)
//   pair: int2 [max(n, n_pages / 2)] pages to copy (source, destination)
//   free: int32 [n_pages] free pages in order (extend, fork); where a page goes (compact)
struct Kv4Ws {
  size_t off = 16, from = 0, pair = 0, free = 0, bytes = 0;
};
inline Kv4Ws kv4_ws(const Kv4& k, int64_t n) {
  auto up = [](size_t b) { return (b + 15) & ~size_t(15); };
  Kv4Ws w;
  const size_t pairs = size_t(n > k.n_pages / 2 ? n : k.n_pages / 2);
  w.from = up(w.off + size_t(n + 1) * 8);
  w.pair = up(w.from + size_t(n) * 4);
  w.free = up(w.pair + pairs * 8);
  w.bytes = up(w.free + size_t(k.n_pages) * 4);
  return w;
}

// Bytes of the attention's partial results (nt_kv4_attn.cu).
size_t kv4_attn_ws_bytes(int n_heads, int n_kv, int hd);

// ------------------------------------------------------------ device helpers --

__device__ __forceinline__ void kv4_flag(const Kv4& k, uint32_t bits) { atomicOr(k.error, bits); }

// Every kernel of the row and page operators is launched so that it may start while the one before it in the
// stream ends, and lets the next one start: it touches memory only after that one has
// ended and its writes are visible.
__device__ __forceinline__ void kv4_dependent() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
}
template <class K, class... A>
inline cudaError_t kv4_launch_smem(K kern, unsigned grid, unsigned block, size_t smem, cudaStream_t s, A... args) {
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
inline cudaError_t kv4_launch(K kern, unsigned grid, unsigned block, cudaStream_t s, A... args) {
  return kv4_launch_smem(kern, grid, block, 0, s, args...);
}

// Rows of a call (include/nt.h, nt_kv4_append).
struct Kv4Rows {
  int32_t layer, n, n_rows, units, checks;
  const int32_t* seq;
  const int32_t* begin;
  int64_t row_stride, head_stride;
};

// What a warp (8-bit cache: a CTA) works on: positions [first, last) of the chunk (page) at position p0 of
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

// Unit u of the call: a chunk of `len` positions (16; 8-bit cache: a page) that entry i's rows may touch.  Entry i's units start
// at begin[i] / len + 2 i: r rows touch at most r / len + 2 chunks, so they do not
// meet entry i + 1's; the units between belong to nobody.  Without `begin` a unit is an
// entry.  false: nothing to do.
// All lanes call it and get the same.
__device__ __forceinline__ bool kv4_span(const Kv4& c, const Kv4Rows& a, int u, Kv4Span* sp, const int len = kKv4Chunk) {
  const int lane = threadIdx.x & 31;
  int i = u, b0 = u, b1 = u + 1, start = u;
  if (a.begin) {
    int lo = 0, hi = a.n;   // entry lo .. hi - 1 has unit u (if any has)
    int step = 1;
    while (step * 32 < hi) step *= 32;
    for (; step; step /= 32) {   // 32 candidates at a time
      const int e = lo + lane * step;
      const bool before = e < hi && a.begin[e] / len + 2 * e <= u;
      const uint32_t m = __ballot_sync(0xffffffffu, before);
      if (!m) return false;
      lo += (31 - __clz(m)) * step;
      hi = lo + step < hi ? lo + step : hi;
    }
    i = lo;
    b0 = a.begin[i];
    b1 = a.begin[i + 1];
    start = b0 / len + 2 * i;
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
  if (u - start > rows / len + 1) return false;   // behind the entry's last chunk (n may be 2^31 - 256: more would not fit an int)
  const int p0 = (n - rows) / len * len + (u - start) * len;   // the chunk's first position
  if (p0 >= n) return false;
  const int first = p0 > n - rows ? p0 : n - rows;
  sp->s = s;
  sp->p0 = p0;
  sp->row = b0 + first - (n - rows);
  sp->first = first - p0;
  sp->last = n - p0 < len ? n - p0 : len;
  return true;
}

// Units of a call (see kv4_span), at most 2^26, so that begin / len + 2 i and the grid
// fit 31 bits (0: n or n_rows is out of range).
inline int32_t kv4_units(int32_t n, int32_t n_rows, const int32_t* begin, int len = kKv4Chunk) {
  const int64_t u = begin ? int64_t(n_rows) / len + 2 * int64_t(n) + 1 : (n < n_rows ? n : n_rows);
  return n < 0 || n_rows < 0 || u > (1 << 26) ? 0 : int32_t(u);
}

// CTAs that look over the entries.
inline int32_t kv4_checks(int32_t n, int32_t n_rows, const int32_t* begin) {
  return begin ? int32_t((int64_t(n) + kKv4CheckEntries - 1) / kKv4CheckEntries) : n > n_rows;
}

// Host checks of a row call's arguments; bytes from the first to the last element of
// the rows (-1: beyond 2^60); whether a (row, kv head) vector of one tensor shares
// bytes with one of another of the same strides that starts d bytes further (same:
// the tensor itself, each vector apart from itself).
nt_status kv4_rows_check(const char* who, const Kv4& k, const Kv4Rows& a, nt_qtype type, const void* pk, const void* pv);
int64_t kv4_rows_bytes(const Kv4& k, const Kv4Rows& a, nt_qtype type);
bool kv4_rows_meet(const Kv4& k, const Kv4Rows& a, int64_t es, int64_t d, bool same);
// A list of n int32 on the device: aligned, and apart from the cache and the workspace.
nt_status kv4_array_check(const Kv4& k, const char* who, const void* p, int64_t n, bool nullable, const void* ws,
                          size_t ws_bytes);
// Flags sequences listed twice.
cudaError_t kv4_launch_listed_twice(const Kv4& k, int32_t n, const int32_t* seq, cudaStream_t s);

// The page operators (include/nt.h) on a checked cache.
nt_status kv4_extend(const char* who, const Kv4& k, int32_t n, const int32_t* seq, const int32_t* count, void* ws,
                     size_t ws_bytes, void* stream);
nt_status kv4_fork(const char* who, const Kv4& k, int32_t n, const int32_t* src, const int32_t* dst, const int32_t* keep,
                   void* ws, size_t ws_bytes, void* stream);
nt_status kv4_free(const char* who, const Kv4& k, int32_t n, const int32_t* seq, const int32_t* keep, void* stream);
nt_status kv4_copy_pages(const char* who, const Kv4& k, int32_t n, const int32_t* src, const int32_t* dst, void* stream);
nt_status kv4_compact(const char* who, const Kv4& k, int32_t* table_out, int32_t* refs_out, int32_t* live, void* ws,
                      size_t ws_bytes, void* stream);

// ---- bulk copies into shared memory, counted on mbarriers of one arrival
__device__ __forceinline__ uint32_t kv4_smem(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void kv4_bar_init(uint32_t bar, uint32_t arrivals = 1) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(arrivals) : "memory");
}
__device__ __forceinline__ void kv4_bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Chunks from global to shared memory, their bytes counted on bar.
__device__ __forceinline__ void kv4_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void kv4_bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Waits for the phase of `parity` to complete, at most kKv4WaitTries tries (each
// of which the hardware may hold for a while); false: gave up.
constexpr int kKv4WaitTries = 1 << 20;
__device__ __forceinline__ bool kv4_bar_wait(uint32_t bar, uint32_t parity) {
  for (int i = 0; i < kKv4WaitTries; i++) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
  }
  return false;
}

// ---- tcgen05
__device__ __forceinline__ void kv4_tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// One thread of a converged warp.  elect.sync, not a test of the thread's number: behind it the compiler knows that one thread
// runs, and issues a product in 9 cycles instead of 45.
__device__ __forceinline__ bool kv4_elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void kv4_tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void kv4_tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

}  // namespace nt
