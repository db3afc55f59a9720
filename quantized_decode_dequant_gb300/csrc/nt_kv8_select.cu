// nt_kv8_select.cu -- which pages of the 8-bit cache a query attends to (include/nt.h,
// nt_kv8_select).
//
// The mathematics.  Per dimension, a head's product with any key of the page is at
// most max(w lo, w hi), which is w hi where w > 0 and w lo where it is not: summed over a kv head's query
// heads that is hi . sum of the positive w plus lo . sum of the negative ones, so the
// heads are added up before any page is looked at and a page costs 2 hd multiplications whatever
// the number of heads.  All are whole numbers: |w| <= 63, 16 heads, 128 dimensions, |lo|, |hi| <= 127 stay below 2^24.
#include "nt_kv8.cuh"

namespace nt {

struct Kv8SelectArgs {
  int32_t layer, n, G, k, first, last, splits;
  const int32_t* seq;
  const int32_t* ctx;
  const float* q;
  int64_t q_stride;
  uint32_t* keys;       // [n][n_kv][max_pages]
  int32_t* out;         // [n][n_kv][k]
};

size_t kv8_select_ws_bytes(const Kv4& k, int64_t n) { return (size_t(n) * k.n_kv * k.max_pages * 4 + 15) / 16 * 16; }

// Sequence of entry i and the positions that it sees (-1: cannot be read, the bit in *bad).
__device__ __forceinline__ int2 kv8_entry(const Kv4& c, const int32_t* seq, const int32_t* ctx, int i, uint32_t* bad) {
  const int s = seq ? seq[i] : i;
  *bad = NT_KV4_BAD_SEQ;
  if (s < 0 || s >= c.max_seqs) return make_int2(-1, 0);
  const int len = c.len[s], n = ctx ? ctx[i] : len;
  *bad = len < 0 || len > c.capacity() || n < 0 || n > len ? NT_KV4_BAD_LEN : 0;
  return make_int2(*bad ? -1 : s, *bad ? 0 : n);
}

constexpr int kKv8ScoreThreads = 256;

// Keys of the pages of (entry, kv head) blockIdx.x / a.splits: whole numbers in the order of the scores.
template <int HD>
__global__ void __launch_bounds__(kKv8ScoreThreads) k_kv8_scores(Kv4 c, Kv8SelectArgs a) {
  constexpr int NT = kKv8ScoreThreads, kLanes = HD / 4;   // lanes of a page, 8 bytes each
  __shared__ int16_t s_w[2 * HD];                         // for lo: sums of the negative w; for hi: of the positive ones
  __shared__ float s_top[NT / 32];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int64_t item = blockIdx.x / a.splits;
  const int split = int(blockIdx.x % a.splits), i = int(item / c.n_kv), g = int(item % c.n_kv);
  kv4_dependent();
  uint32_t bad;
  const int2 e = kv8_entry(c, a.seq, a.ctx, i, &bad);
  if (bad) {
    if (t == 0 && split == 0) kv4_flag(c, bad);
    return;
  }
  const int m = (int64_t(e.y) + c.page_len - 1) / c.page_len;
  if (m <= a.k) return;
  const float* q = a.q + int64_t(i) * a.q_stride + int64_t(g) * a.G * HD;
  float top = 0.f;
  for (int x = t; x < a.G * HD; x += NT) {
    const float y = fabsf(q[x]);
    if (y < INFINITY) top = fmaxf(top, y);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NT / 32; w++) top = fmaxf(top, s_top[w]);
  // 63 is 1.96875 2^5: f = exponent - 5, one more above 1.96875
  int f = 0;
  if (top > 0.f) {
    const float up = top < 0x1p-100f ? top * 0x1p60f : top;
    const uint32_t b = __float_as_uint(up);
    f = int(b >> 23) - 132 + ((b & 0x7fffffu) > 0x7c0000u) - (top < 0x1p-100f ? 60 : 0);
  }
  if (t < HD) {
    int pos = 0, neg = 0;
    for (int h = 0; h < a.G; h++) {
      const float x = q[h * HD + t];
      int w = 0;
      if (fabsf(x) < INFINITY) w = __float2int_rn(scalbnf(x, -f));
      else if (x == x) w = x > 0.f ? 63 : -63;
      if (w > 0) pos += w; else neg += w;
    }
    s_w[t] = int16_t(neg);
    s_w[HD + t] = int16_t(pos);
  }
  __syncthreads();
  const int sub = lane % kLanes;
  int w[4];
#pragma unroll
  for (int y = 0; y < 4; y++) w[y] = reinterpret_cast<const int*>(s_w)[4 * sub + y];
  const Kv8Page L(c);
  const uint8_t* pool = c.pool + int64_t(a.layer) * c.n_pages * c.page_bytes();
  const int32_t* row = c.table + int64_t(e.x) * c.max_pages;
  uint32_t* keys = a.keys + item * c.max_pages;
  constexpr int kPer = 32 / kLanes;                       // pages of a warp at a time
  const int step = a.splits * (NT / 32) * kPer;
  for (int j0 = (split * (NT / 32) + warp) * kPer; j0 < m; j0 += step) {
    const int j = j0 + lane / kLanes;
    int page = j < m ? row[j] : -1, sum = 0, ex = 0;
    if (page < 0 || page >= c.n_pages) {
      if (j < m && sub == 0) kv4_flag(c, NT_KV4_BAD_PAGE);
      page = -1;
    }
    if (page >= 0) {
      const uint8_t* at = pool + page * c.page_bytes() + L.exps(g);
      const uint2 b = *reinterpret_cast<const uint2*>(at + 16 + 8 * sub);
      ex = *reinterpret_cast<const int8_t*>(at);
      sum = __dp2a_lo(w[0], int(b.x), 0);
      sum = __dp2a_hi(w[1], int(b.x), sum);
      sum = __dp2a_lo(w[2], int(b.y), sum);
      sum = __dp2a_hi(w[3], int(b.y), sum);
    }
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (j < m && sub == 0) {
      const uint32_t s = __float_as_uint(float(sum) * kv8_exp2i(ex));
      const uint32_t key = s >> 31 ? ~s : s | 0x80000000u;
      keys[j] = j < a.first || j >= m - a.last ? 0xffffffffu : key;   // (no score has the key 0xffffffff)
    }
  }
}

constexpr int kKv8PickThreads = 512;

// The places of the a.k largest keys of (entry, kv head) blockIdx.x, the lower place
// first among equals, ascending: the a.k-th largest key digit by digit from counts, then one pass
// that writes what is above it and the first of those equal to it.
__global__ void __launch_bounds__(kKv8PickThreads) k_kv8_pick(Kv4 c, Kv8SelectArgs a) {
  constexpr int NT = kKv8PickThreads;
  __shared__ int s_count[256], s_part[2][NT / 32], s_digit, s_left;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int64_t item = blockIdx.x;
  kv4_dependent();
  uint32_t bad;
  const int2 e = kv8_entry(c, a.seq, a.ctx, int(item / c.n_kv), &bad);
  const int m = (int64_t(e.y) + c.page_len - 1) / c.page_len;
  int32_t* out = a.out + item * a.k;
  if (m <= a.k) {
    for (int j = t; j < a.k; j += NT) out[j] = j < m ? j : -1;
    return;
  }
  const uint32_t* keys = a.keys + item * c.max_pages;
  uint32_t prefix = 0u;
  int left = a.k;                                        // of those whose upper digits are prefix's
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int x = t; x < 256; x += NT) s_count[x] = 0;
    __syncthreads();
    for (int j = t; j < m; j += NT) {
      const uint32_t key = keys[j];
      if (shift == 24 || (key ^ prefix) >> (shift + 8) == 0u) atomicAdd(&s_count[key >> shift & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {                                     // lane x has digits 255 - 8 x and the 7 below
      int mine = 0;
#pragma unroll
      for (int y = 0; y < 8; y++) mine += s_count[255 - 8 * lane - y];
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += z;
      }
      int before = upto - mine;
      if (before < left && upto >= left)
        for (int y = 0; y < 8; y++) {
          const int d = 255 - 8 * lane - y, n = s_count[d];
          if (before < left && before + n >= left) {
            s_digit = d;
            s_left = left - before;
          }
          before += n;
        }
    }
    __syncthreads();
    prefix |= uint32_t(s_digit) << shift;
    left = s_left;
    __syncthreads();
  }
  int above = 0, equal = 0;                              // of the places before this round's
  for (int j0 = 0; j0 < m; j0 += NT) {
    const int j = j0 + t;
    const uint32_t key = j < m ? keys[j] : 0u;
    const bool over = j < m && key > prefix, same = j < m && key == prefix;
    const uint32_t mo = __ballot_sync(0xffffffffu, over), ms = __ballot_sync(0xffffffffu, same);
    if (lane == 0) {
      s_part[0][warp] = __popc(mo);
      s_part[1][warp] = __popc(ms);
    }
    __syncthreads();
    int po = above, ps = equal, ao = 0, as = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; w++) {
      if (w < warp) { po += s_part[0][w]; ps += s_part[1][w]; }
      ao += s_part[0][w];
      as += s_part[1][w];
    }
    po += __popc(mo & ((1u << lane) - 1u));
    ps += __popc(ms & ((1u << lane) - 1u));
    if (over) out[po + (ps < left ? ps : left)] = j;
    if (same && ps < left) out[po + ps] = j;
    above += ao;
    equal += as;
    __syncthreads();
  }
}

}  // namespace nt

using namespace nt;

extern "C" nt_status nt_kv8_select(const nt_kv8_cache* c, int32_t layer, int32_t n_heads, int32_t n, const int32_t* dev_seq,
                                   const int32_t* dev_ctx, const float* dev_q, int64_t q_stride, int32_t n_select,
                                   int32_t n_first, int32_t n_last, int32_t* dev_pages, void* dev_workspace,
                                   size_t workspace_bytes, void* stream) {
  const char* who = "nt_kv8_select";
  auto bad = [&](const char* what) { return fail(NT_E_INVAL, std::string(who) + ": " + what); };
  Kv4 k;
  nt_status st = kv8_check(c, who, true, &k);
  if (st) return st;
  if (layer < 0 || layer >= k.n_layers) return bad("layer out of range");
  if (n_heads < 1 || n_heads % k.n_kv) return bad("n_heads must be a positive multiple of n_kv_heads");
  if (n_heads / k.n_kv > kKv8MaxGroup) return fail(NT_E_UNSUPPORTED, std::string(who) + ": more than 16 query heads per kv head");
  if (n < 0 || n > 65536 || (!dev_seq && n > k.max_seqs)) return bad("n out of range");
  if (n_select < 1 || n_select > 65536) return bad("n_select outside [1, 65536]");
  if (n_first < 0 || n_last < 0 || int64_t(n_first) + n_last > n_select) return bad("n_first and n_last must not be negative, their sum at most n_select");
  const int64_t row = int64_t(n_heads) * k.hd;
  if (q_stride < row || q_stride % 4 || q_stride > (int64_t(1) << 40)) return bad("q_stride must be a multiple of 4 and at least n_heads * head_dim");
  if (!kv4_aligned(dev_q, 16) || !kv4_aligned(dev_workspace, 16)) return bad("q or workspace is NULL or not 16-byte aligned");
  if (!kv4_aligned(dev_pages, 4) || (dev_seq && !kv4_aligned(dev_seq, 4)) || (dev_ctx && !kv4_aligned(dev_ctx, 4)))
    return bad("a list is NULL or not 4-byte aligned");
  const size_t wb = kv8_select_ws_bytes(k, n);
  if (workspace_bytes < wb) return bad("workspace too small");
  const int64_t items = int64_t(n) * k.n_kv;
  if (items > (1 << 24)) return bad("n * n_kv_heads above 2^24");
  if (n == 0) return NT_OK;
  const int64_t qb = ((n - 1) * q_stride + row) * 4, ob = items * n_select * 4, lb = int64_t(n) * 4;
  auto meets = [&](const void* p, int64_t bytes) {   // a written buffer and everything else
    return kv4_meets_cache(k, p, bytes) || kv4_overlap(p, bytes, dev_q, qb) || (dev_seq && kv4_overlap(p, bytes, dev_seq, lb)) ||
           (dev_ctx && kv4_overlap(p, bytes, dev_ctx, lb));
  };
  if (meets(dev_pages, ob) || meets(dev_workspace, int64_t(wb)) || kv4_overlap(dev_pages, ob, dev_workspace, int64_t(wb)))
    return bad("the output or the workspace overlaps another buffer");
  Kv8SelectArgs a{layer, n, n_heads / k.n_kv, n_select, n_first, n_last, 1, dev_seq, dev_ctx, dev_q, q_stride,
                        static_cast<uint32_t*>(dev_workspace), dev_pages};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (k.max_pages > n_select) {
    const int64_t rounds = (k.max_pages + 8 * 4 - 1) / (8 * 4);       // four pages a warp
    const int64_t splits = 152 * 4 / items;
    a.splits = int32_t(splits < 1 ? 1 : (splits > rounds ? rounds : splits));
    const unsigned grid = unsigned(items * a.splits);
    NT_CUDA(k.hd == 64 ? kv4_launch(k_kv8_scores<64>, grid, unsigned(kKv8ScoreThreads), s, k, a)
                       : kv4_launch(k_kv8_scores<128>, grid, unsigned(kKv8ScoreThreads), s, k, a));
  }
  NT_CUDA(kv4_launch(k_kv8_pick, unsigned(items), unsigned(kKv8PickThreads), s, k, a));
  return NT_OK;
}
