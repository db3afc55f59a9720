// nt_kv4_attn.cuh -- what the two kernels of attention over the paged 4-bit cache
// share: arguments, decoding, the share-out of the work and the merge of partial results.
#pragma once

#include "nt_kv4.cuh"

namespace nt {

constexpr int kKv4Batch = 1024;        // sequences of one launch: their pair offsets are kept in shared memory
constexpr int kKv4AttnMaxCtas = 152;   // one CTA per SM; the workspace holds two partial results of each

struct Kv4AttnArgs {
  int32_t layer, n, G;
  int32_t seq0;                        // sequence of entry 0 where none are listed
  const int32_t* seq;
  const float* q;
  int64_t q_stride;
  float* out;
  int64_t out_stride;
  float q_scale;                       // 8 log2(e) / sqrt(hd): what q is multiplied by on top of a power of two
  float* part;                         // [CTA][2] partial results
};

// The attention kernel on tcgen05 (nt_kv4_attn_tc.cu): 128 dimensions, G 8 or 16; *ctas: its CTAs.  Whether it can run is asked
// first: not where it was compiled for other registers than it shares out (as for a debugger).
bool kv4_attn_tc_runs(int G);
cudaError_t kv4_launch_attn_tc(const Kv4& k, const Kv4AttnArgs& a, cudaStream_t s, int* ctas);

// Partial result of one item: o [rows][HD], then (reference m, sum l) per row, then
// a header of 4 words (used by the CTAs' slot 1: the item, -1 none, and the
// number of CTAs that worked on it).
__host__ __device__ constexpr int kv4_part_floats(int hd, int rows) { return rows * hd + 2 * rows + 4; }

// ------------------------------------------------------------ small pieces --

__device__ __forceinline__ float kv4_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint4 kv4_lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 kv4_lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t kv4_lds4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
// NG consecutive words
template <int NG>
__device__ __forceinline__ void kv4_words(uint32_t a, uint32_t (&w)[NG]) {
  if (NG == 4) {
    const uint4 v = kv4_lds16(a);
    w[0] = v.x; w[1] = v.y; w[2 % NG] = v.z; w[3 % NG] = v.w;
  } else {
    const uint2 v = kv4_lds8(a);
    w[0] = v.x; w[1] = v.y;
  }
}
__device__ __forceinline__ uint32_t kv4_h2fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t kv4_h2mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// (w & mask) | magic
template <uint32_t mask>
__device__ __forceinline__ uint32_t kv4_pick(uint32_t w, uint32_t magic) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "n"(mask), "r"(magic));
  return d;
}
// The four half2 of a word: value pairs (code k, code k + 4), k = 0..3, times the
// scale pair d; d72 = -72 d.  (Two of the shifts can be saved by taking codes 0 and
// 2 as 1024 + q, less 1032, times d: measured 4% slower at 131077 positions with
// mma.sync and 2% with tcgen05: as many instructions, more of them half2.)
__device__ __forceinline__ void kv4_decode(uint32_t w, uint32_t d, uint32_t d72, uint32_t (&b)[4]) {
  constexpr uint32_t k64 = 0x54005400u;
  b[0] = kv4_h2fma(kv4_pick<0x00f000f0u>(w << 4, k64), d, d72);
  b[1] = kv4_h2fma(kv4_pick<0x00f000f0u>(w, k64), d, d72);
  b[2] = kv4_h2fma(kv4_pick<0x00f000f0u>(w >> 4, k64), d, d72);
  b[3] = kv4_h2fma(kv4_pick<0x00f000f0u>(w >> 8, k64), d, d72);
}
constexpr uint32_t kMinus72 = 0xd480d480u;   // f16 -72 twice

// the low or the high half of x twice, as the half2 instructions can take it themselves
__device__ __forceinline__ uint32_t kv4_half(uint32_t x, bool high) {
  uint32_t d;
  if (high) asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(d) : "r"(x));
  else asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(d) : "r"(x));
  return d;
}

// hi and lo f16 terms of two fp32 values
__device__ __forceinline__ void kv4_split(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x0 - f.x, x1 - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
// Sequence and length of listed entry e (length 0 and *bad where it cannot be read).
__device__ __forceinline__ int2 kv4_entry(const Kv4& c, const Kv4AttnArgs& a, int e, uint32_t* bad) {
  const int s = a.seq ? a.seq[e] : a.seq0 + e;
  *bad = NT_KV4_BAD_SEQ;
  if (s < 0 || s >= c.max_seqs) return make_int2(-1, 0);
  const int n = c.len[s];
  *bad = n < 0 || n > c.capacity() ? NT_KV4_BAD_LEN : 0;
  return make_int2(*bad ? -1 : s, *bad ? 0 : n);
}
// Entry of prefix (ascending, prefix[0] = 0) that holds chunk x: prefix[i] <= x < prefix[i + 1].
__device__ __forceinline__ int kv4_find(const int* prefix, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Units of the entries, item after item: an entry has one item per kv head, an item
// its positions / unit_len units and `cost` more; prefix[e] is the first unit of
// entry e, prefix[n] all of them.  Every thread of the CTA calls it; afterwards its own
// warp may read prefix and entry.  sums: NW ints of shared memory.
template <int NW>
__device__ __forceinline__ void kv4_count(const Kv4& c, const Kv4AttnArgs& a, int unit_len, int cost, int* prefix, int2* entry,
                                          int* sums) {
  constexpr int kFew = 128;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, n = a.n;
  auto units = [&](int len) { return len ? ((len + unit_len - 1) / unit_len + cost) * c.n_kv : 0; };
  if (n <= kFew) {   // every warp for itself, all to the same places: no barrier
    int2 sl[kFew / 32];
#pragma unroll
    for (int i = 0; i < kFew / 32; i++) {
      const int e = 32 * i + lane;
      uint32_t bad = 0;
      sl[i] = make_int2(-1, 0);
      if (e < n) sl[i] = kv4_entry(c, a, e, &bad);
      if (bad && blockIdx.x == 0 && warp == 0) kv4_flag(c, bad);
    }
    int run = 0;
#pragma unroll
    for (int i = 0; i < kFew / 32; i++) {
      if (32 * i >= n) break;
      const int e = 32 * i + lane, mine = units(sl[i].y);
      int x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (e < n) {
        entry[e] = sl[i];
        prefix[e] = run + x - mine;
      }
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) prefix[n] = run;
    __syncwarp();
    return;
  }
  int run = 0;
  for (int e0 = 0; e0 < n; e0 += 32 * NW) {
    const int e = e0 + t;
    int mine = 0;
    if (e < n) {
      uint32_t bad;
      const int2 sl = kv4_entry(c, a, e, &bad);
      if (bad && blockIdx.x == 0) kv4_flag(c, bad);
      entry[e] = sl;
      mine = units(sl.y);
    }
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < NW && e0 + 32 * w < n; w++) {
      const int y = sums[w];
      if (w < warp) before += y;
      all += y;
    }
    if (e < n) prefix[e] = run + before + x - mine;
    run += all;
    __syncthreads();
  }
  if (t == 0) prefix[n] = run;
  __syncthreads();
}

// The entries without a position: zeros, or NaN where they cannot be read.
__device__ __forceinline__ void kv4_empty_entries(const Kv4& c, const Kv4AttnArgs& a, const int2* entry, int hd) {
  for (int e = blockIdx.x; e < a.n; e += gridDim.x)
    if (entry[e].y == 0)
      for (int x = threadIdx.x; x < c.n_kv * a.G * hd; x += blockDim.x)
        a.out[int64_t(e) * a.out_stride + x] = entry[e].x < 0 ? NAN : 0.f;
}

// Merges the partial results that a CTA's warps left in SLOTS slots (slot_item: the
// item, -1 none; slots of an item follow one another), a warp per head and a lane per
// slot, in the slots' order.  range(item, first, units): the item's units, those of
// this CTA being [c0, c1).  An item that lies within them is written out; one that does not leaves
// a partial result at part0 (begun before) or behind it (begun here: the header says
// which item and how many CTAs of `span` units it has; NULL: at part0 always).  order:
// 32 ints of the warp.
template <int HD, int ROWS, int NW, int SLOTS, class P, class R>
__device__ __forceinline__ void kv4_merge(const Kv4& c, const Kv4AttnArgs& a, const int* slot_item, P slot_ptr, int* order,
                                          R range, int c0, int c1, int span, float* part0, int* header) {
  constexpr int V = HD / 32, kPart = kv4_part_floats(HD, ROWS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.G;
  const int mine = lane < SLOTS ? slot_item[lane] : -1;
  int turn = warp;   // (item, head) pairs go round the warps
  for (uint32_t left = __ballot_sync(0xffffffffu, mine >= 0); left; turn = (turn + NW * G - G) % NW) {
    const int a0 = __ffs(left) - 1, item = __shfl_sync(0xffffffffu, mine, a0);
    const uint32_t members = __ballot_sync(0xffffffffu, mine == item);
    left &= ~members;
    const int nm = __popc(members);
    __syncwarp();
    if (mine == item) order[__popc(members & ((1u << lane) - 1u))] = lane;
    __syncwarp();
    const int nth = order[lane < nm ? lane : 0];   // lane i: the item's i-th slot
    int first, units;
    range(item, first, units);
    const bool whole = first >= c0 && first + units <= c1;
    float* part = !header || first < c0 ? part0 : part0 + kPart;
    float* to = whole ? a.out + int64_t(item / c.n_kv) * a.out_stride + int64_t(item % c.n_kv) * G * HD : part;
    for (int h = turn; h < G; h += NW) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < nm) ml = reinterpret_cast<const float2*>(slot_ptr(nth) + ROWS * HD)[h];
      float M = ml.x;
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      float f = lane < nm ? kv4_ex2(ml.x - M) : 0.f, sum = ml.y * f;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (whole) f /= sum;
      float o[V];
#pragma unroll
      for (int v = 0; v < V; v++) o[v] = 0.f;
#pragma unroll 1
      for (int i = 0; i < nm; i += 4) {
#pragma unroll
        for (int u = 0; u < 4; u++) {
          const int w = __shfl_sync(0xffffffffu, nth, i + u);
          const float fw = __shfl_sync(0xffffffffu, f, i + u);
          const float* r = slot_ptr(w) + h * HD + V * lane;
          if (i + u >= nm) continue;
          if (V == 4) {
            const float4 x = *reinterpret_cast<const float4*>(r);
            o[0] = fmaf(x.x, fw, o[0]); o[1] = fmaf(x.y, fw, o[1]);
            o[2 % V] = fmaf(x.z, fw, o[2 % V]); o[3 % V] = fmaf(x.w, fw, o[3 % V]);
          } else {
            const float2 x = *reinterpret_cast<const float2*>(r);
            o[0] = fmaf(x.x, fw, o[0]); o[1] = fmaf(x.y, fw, o[1]);
          }
        }
      }
      if (V == 4) *reinterpret_cast<float4*>(to + h * HD + V * lane) = make_float4(o[0], o[1], o[2 % V], o[3 % V]);
      else *reinterpret_cast<float2*>(to + h * HD + V * lane) = make_float2(o[0], o[1]);
      if (!whole && lane == 0) reinterpret_cast<float2*>(part + ROWS * HD)[h] = make_float2(M, sum);
    }
    if (header && !whole && first >= c0 && threadIdx.x == 0) {   // begun here: k_kv4_attn_merge collects it from here
      header[1] = (first + units - 1) / span - int(blockIdx.x) + 1;
      header[0] = item;
    }
  }
}

}  // namespace nt
