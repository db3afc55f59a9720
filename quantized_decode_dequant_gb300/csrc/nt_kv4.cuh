// nt_kv4.cuh -- layout, argument checks and workspace of the paged 4-bit K/V
// cache (include/nt.h, nt_kv4_cache), shared by its operators (nt_kv4.cu) and
// the attention over it (nt_kv4_attn.cu).
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

  __host__ __device__ int64_t page_bytes() const { return int64_t(n_kv) * (page_len / kKv4Chunk) * kv4_chunk_bytes(hd); }
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

}  // namespace nt
