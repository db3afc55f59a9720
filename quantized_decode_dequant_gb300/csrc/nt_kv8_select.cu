// nt_kv8_select.cu -- which pages of the 8-bit cache a query attends to (include/nt.h,
// nt_kv8_select).
//
// The mathematics.  Per dimension, a head's product with any key of the page is at most max(w lo, w hi), which is w hi
// where w > 0 and w lo where it is not: summed over a kv head's query heads that is hi . sum of the positive w plus
// lo . sum of the negative ones, so the heads are added up before any page is looked at and a page costs 2 hd
// multiplications whatever the number of heads.  All are whole numbers: |w| <= 63, 16 heads, 128 dimensions,
// |lo|, |hi| <= 127 stay below 2^24.
//
// What bounds it: for one long sequence latency (2049 pages, 8 kv heads, 4.5 MB: 8.0 us, of which the choice of 64 is 3.9 and
// a launch, the table and the bounds one after the other the rest); for many, reads of 272 bytes, which eight
// clusters make of a page's 2176 since an item is one kv head (24 x 30k positions, 25 MB: 13.8 us, 1.8 TB/s).
#include "nt_kv8.cuh"

namespace nt {

struct Kv8SelectArgs {
  int32_t layer, n, G, k, first, last;
  int32_t seq0;         // sequence of entry 0 where none are listed
  const int32_t* seq;
  const int32_t* ctx;
  const float* q;
  int64_t q_stride;
  uint32_t* keys;       // [n][n_kv][kv8_key_stride]
  int32_t* out;         // [n][n_kv][k]
};

__host__ __device__ __forceinline__ int64_t kv8_key_stride(const Kv4& k) { return (int64_t(k.max_pages) + 3) / 4 * 4; }
size_t kv8_select_ws_bytes(const Kv4& k, int64_t n) { return size_t(n) * k.n_kv * kv8_key_stride(k) * 4; }

constexpr int kKv8SelectThreads = 256;
constexpr int kKv8ScorePages = 16;   // of a warp at a time
constexpr int kKv8PickBins = 1024;

// The places of the k largest of an item's m keys, the lower place first among equals, ascending, by a whole CTA.  A thread has m / 256
// keys side by side, in its registers where there are no more than 4096 in all.  The k-th largest is found by counting keys in 1024 bins of
// equal width between the least and the largest, then in the bin where it lies, and so on; as soon as all keys of
// that bin are wanted they and those above are the choice.  (Bins of the keys' upper bits, which few scores differ in, had all
// threads count in the same few: 8.7 us for 2049 keys; candidates bit by bit with a count of all keys each: 12.5; 16 keys for each of the first
// threads: 4.6, this 3.9.)
__device__ __forceinline__ void kv8_pick(const uint32_t* keys, int m, int k, int32_t* out) {
  constexpr int NT = kKv8SelectThreads, NW = NT / 32, R = 16, kBins = kKv8PickBins, kOwn = kBins / NT;
  __shared__ __align__(16) int s_bins[2][kBins];
  __shared__ uint32_t s_part[4][NW];
  __shared__ int s_bin, s_left, s_in;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  constexpr uint32_t kAlways = 0xffffffffu;
  const int chunk = R * NT, per = m < chunk ? (m + NT - 1) / NT : R;     // keys of a thread in a round of NT * per
  uint32_t key[R];
  auto get = [&](int j0) {                               // keys j0 + per t ..; behind the end zeros
#pragma unroll
    for (int y = 0; y < R; y++) {
      const int j = j0 + per * t + y;
      key[y] = y < per && j < m ? keys[j] : 0u;
    }
  };
  auto each = [&](auto f) {                              // f(key, whether it is one) for all of this thread's
    for (int j0 = 0; j0 < m; j0 += NT * per) {
      if (m > chunk) get(j0);
#pragma unroll
      for (int y = 0; y < R; y++)
        if (y < per) f(key[y], j0 + per * t + y < m);
    }
  };
  get(0);
  *reinterpret_cast<int4*>(&s_bins[0][4 * t]) = make_int4(0, 0, 0, 0);
  uint32_t least = kAlways, most = 0u, always = 0u;      // of the keys that are not always taken, and how many are
  each([&](uint32_t x, bool is) {
    const bool taken = is && x == kAlways;
    always += taken;
    if (is && !taken) {
      least = min(least, x);
      most = max(most, x);
    }
  });
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  always = __reduce_add_sync(0xffffffffu, always);
  if (lane == 0) { s_part[0][warp] = least; s_part[1][warp] = most; s_part[2][warp] = always; }
  __syncthreads();
  least = __reduce_min_sync(0xffffffffu, s_part[0][lane % NW]);
  most = __reduce_max_sync(0xffffffffu, s_part[1][lane % NW]);
  always = __reduce_add_sync(0xffffffffu, lane < NW ? s_part[2][lane] : 0u);
  // keys from `base` on, 2^width of them, are looked at; those above are taken, `left` of these are
  uint32_t base = least;
  int width = 32 - __clz(most - least), left = k - int(always);
  bool found = left == 0;                                // (m > k: there are others)
  if (found) base = kAlways;
  for (int buf = 0; !found && width > 0; buf ^= 1) {     // (s_bins[buf] is zero)
    const int shift = width > 10 ? width - 10 : 0;
    const uint32_t bins = 1u << (width - shift);         // (fewer at last: keys further up are taken already)
    each([&](uint32_t x, bool is) {
      const uint32_t bin = (x - base) >> shift;          // (keys below base wrap round to large numbers)
      if (is && x >= base && bin < bins && x != kAlways) atomicAdd(&s_bins[buf][kBins - 1 - bin], 1);   // the largest keys first
    });
    *reinterpret_cast<int4*>(&s_bins[buf ^ 1][4 * t]) = make_int4(0, 0, 0, 0);
    __syncthreads();
    const int4 own = *reinterpret_cast<const int4*>(&s_bins[buf][kOwn * t]);
    const int n[kOwn] = {own.x, own.y, own.z, own.w}, mine = own.x + own.y + own.z + own.w;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += z;
    }
    if (lane == 31) s_part[3][warp] = uint32_t(upto);
    __syncthreads();
    int before = upto - mine + int(__reduce_add_sync(0xffffffffu, lane < warp ? s_part[3][lane % NW] : 0u));
    if (before < left && before + mine >= left)
#pragma unroll
      for (int y = 0; y < kOwn; y++) {
        if (before < left && before + n[y] >= left) {
          s_bin = kBins - 1 - (kOwn * t + y);
          s_left = left - before;
          s_in = n[y];
        }
        before += n[y];
      }
    __syncthreads();
    base += uint32_t(s_bin) << shift;
    width = shift;
    left = s_left;
    found = s_in == left;
  }
  const int ties = found ? m : left;                     // of those equal to base, how many are taken
  int taken = 0, equal = 0;                              // of the places before this pass over them
  for (int j0 = 0; j0 < m; j0 += NT * per) {
    if (m > chunk) get(j0);
    int over = 0, same = 0;
#pragma unroll
    for (int y = 0; y < R; y++) {
      const bool in = y < per && j0 + per * t + y < m;
      over += in && key[y] > base;
      same += in && key[y] == base;
    }
    int both = over | same << 16;                        // (4096 at most)
    const int own = both;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, both, o);
      if (lane >= o) both += z;
    }
    __syncthreads();
    if (lane == 31) s_part[1][warp] = uint32_t(both);
    __syncthreads();
    const uint32_t w = s_part[1][lane % NW];
    both += int(__reduce_add_sync(0xffffffffu, lane < warp ? w : 0u)) - own;
    const int all = int(__reduce_add_sync(0xffffffffu, lane < NW ? w : 0u));
    int po = taken + (both & 0xffff), ps = equal + (both >> 16);   // those above base, and equal to it, before this thread's
    if (over + same)
#pragma unroll
      for (int y = 0; y < R; y++) {
        const int j = j0 + per * t + y;
        if (y >= per || j >= m) continue;
        if (key[y] > base) { out[po + min(ps, ties)] = j; po++; }
        if (key[y] == base) {
          if (ps < ties) out[po + ps] = j;
          ps++;
        }
      }
    taken += all & 0xffff;
    equal += all >> 16;
  }
}

// A cluster per (entry, kv head): its CTAs share out the pages' scores, the first one picks.  Keys are whole numbers in the order of the scores.  A
// warp takes 16 pages at a time, eight lanes each; their places in the pool are looked up a round ahead.  (As two launches, with
// the same code: 1 x 131k 8.5 us, 24 x 30k 16.3.)
template <int HD>
__global__ void __launch_bounds__(kKv8SelectThreads) k_kv8_select(Kv4 c, Kv8SelectArgs a) {
  constexpr int NT = kKv8SelectThreads, NW = NT / 32, kRun = 16, kRuns = 2 * HD / (8 * kRun);   // runs of 16 bounds of a lane: hd 128: one of lo, one of hi
  __shared__ __align__(16) int16_t s_w[2 * HD];           // for lo: sums of the negative w; for hi: of the positive ones
  __shared__ float s_top[NW];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int64_t item = blockIdx.y;
  const int split = int(blockIdx.x), splits = int(gridDim.x), i = int(item / c.n_kv), g = int(item % c.n_kv);
  kv4_dependent();
  // the queries are on the way while the entry is looked up
  const float* q = a.q + int64_t(i) * a.q_stride + int64_t(g) * a.G * HD;
  float top = 0.f;
  for (int x = 4 * t; x < a.G * HD; x += 4 * NT) {
    const float4 y = *reinterpret_cast<const float4*>(q + x);
    auto size = [](float z) { return fabsf(z) < INFINITY ? fabsf(z) : 0.f; };
    top = fmaxf(top, fmaxf(fmaxf(size(y.x), size(y.y)), fmaxf(size(y.z), size(y.w))));
  }
  uint32_t bad;
  const int2 e = kv8_entry(c, a.seq, a.ctx, a.seq0, i, &bad);
  if (bad && t == 0 && split == 0) kv4_flag(c, bad);
  const int m = int((int64_t(e.y) + c.page_len - 1) / c.page_len);
  int32_t* out = a.out + item * a.k;
  if (m <= a.k) {                                         // (the whole cluster; m is 0 where the entry cannot be read)
    for (int j = split * NT + t; j < a.k; j += splits * NT) out[j] = j < m ? j : -1;
    return;
  }
  const int32_t* row = c.table + int64_t(e.x) * c.max_pages;
  auto look = [&](int j0) { return lane < kKv8ScorePages && j0 + lane < m ? row[j0 + lane] : 0; };
  const int step = splits * NW * kKv8ScorePages;
  int j0 = (split * NW + warp) * kKv8ScorePages, page = j0 < m ? look(j0) : 0;
  // ---- the weights of the group's queries
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; w++) top = fmaxf(top, s_top[w]);
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
  const int sub = lane & 7, of = lane >> 3;               // this lane's part of page `of` of four
  int w[kRuns][kRun / 2];
#pragma unroll
  for (int r = 0; r < kRuns; r++)
#pragma unroll
    for (int y = 0; y < kRun / 2; y++) w[r][y] = reinterpret_cast<const int*>(s_w)[(r * 8 + sub) * (kRun / 2) + y];
  const Kv8Page L(c);
  const uint8_t* heads = c.pool + int64_t(a.layer) * c.n_pages * c.page_bytes() + L.exps(g);
  uint32_t* keys = a.keys + item * kv8_key_stride(c);
  for (; j0 < m; j0 += step) {
    const int next = j0 + step < m ? look(j0 + step) : 0;
    const bool there = lane < kKv8ScorePages && j0 + lane < m, good = page >= 0 && page < c.n_pages;
    if (there && !good) kv4_flag(c, NT_KV4_BAD_PAGE);
    if (!good) page = -1;
    uint4 b[kKv8ScorePages / 4][kRuns];
#pragma unroll
    for (int y = 0; y < kKv8ScorePages / 4; y++) {
      const int p = __shfl_sync(0xffffffffu, page, 4 * y + of);
#pragma unroll
      for (int r = 0; r < kRuns; r++) {
        b[y][r] = make_uint4(0u, 0u, 0u, 0u);
        if (p >= 0 && j0 + 4 * y + of < m) b[y][r] = *reinterpret_cast<const uint4*>(heads + p * c.page_bytes() + 16 + (r * 8 + sub) * kRun);
      }
    }
    int ex = 0;
    if (there && page >= 0) ex = *reinterpret_cast<const int8_t*>(heads + page * c.page_bytes());
    int mine = 0;                                         // the sum of this lane's page
#pragma unroll
    for (int y = 0; y < kKv8ScorePages / 4; y++) {
      int sum = 0;
#pragma unroll
      for (int r = 0; r < kRuns; r++) {
        const uint32_t u[4] = {b[y][r].x, b[y][r].y, b[y][r].z, b[y][r].w};
#pragma unroll
        for (int z = 0; z < 4; z++) {
          sum = __dp2a_lo(w[r][2 * z], int(u[z]), sum);
          sum = __dp2a_hi(w[r][2 * z + 1], int(u[z]), sum);
        }
      }
#pragma unroll
      for (int o = 4; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      sum = __shfl_sync(0xffffffffu, sum, 8 * (lane & 3));
      if (lane >> 2 == y) mine = sum;
    }
    if (there) {
      const int j = j0 + lane;
      const uint32_t z = __float_as_uint(float(mine) * kv8_exp2i(ex)), key = z >> 31 ? ~z : z | 0x80000000u;
      // (0xffffffff is always chosen: n_first + n_last of them and no more, whatever the bytes of a page that was never written)
      keys[j] = j < a.first || j >= m - a.last ? 0xffffffffu : min(key, 0xfffffffeu);
    }
    page = next;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (split == 0) kv8_pick(keys, m, a.k, out);
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
  const Kv8SelectArgs a{layer, n, n_heads / k.n_kv, n_select, n_first, n_last, 0, dev_seq, dev_ctx, dev_q, q_stride,
                        static_cast<uint32_t*>(dev_workspace), dev_pages};
  // a cluster of up to 16 CTAs per item, as far as the GPU holds four CTAs an SM and each has pages to look at (24 x 30k, 192 items, with
  // the attention behind it: 2 an SM 67.2 us, 4: 53.0, 8: 56.5)
  const int64_t per = kKv8SelectThreads / 32 * kKv8ScorePages, rounds = (k.max_pages + per - 1) / per;
  int64_t splits = 152 * 4 / items;
  splits = splits > 16 ? 16 : splits;
  splits = k.max_pages <= n_select || splits < 1 ? 1 : (splits > rounds ? rounds : splits);
  static const cudaError_t wide[2] = {cudaFuncSetAttribute(k_kv8_select<64>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1),
                                      cudaFuncSetAttribute(k_kv8_select<128>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)};
  if (wide[k.hd == 128] != cudaSuccess) return cuda_fail(wide[k.hd == 128], who);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(splits);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(splits), 0u);
  cfg.blockDim = dim3(unsigned(kKv8SelectThreads));
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  constexpr int64_t kMost = 65535;                        // items of a launch
  for (int64_t at = 0; at < n; at += kMost / k.n_kv) {
    Kv8SelectArgs part = a;
    part.n = int32_t(n - at < kMost / k.n_kv ? n - at : kMost / k.n_kv);
    part.seq0 = int32_t(at);
    if (dev_seq) part.seq += at;
    if (dev_ctx) part.ctx += at;
    part.q += at * q_stride;
    part.keys += at * k.n_kv * kv8_key_stride(k);
    part.out += at * k.n_kv * n_select;
    cfg.gridDim.y = unsigned(int64_t(part.n) * k.n_kv);
    NT_CUDA(k.hd == 64 ? cudaLaunchKernelEx(&cfg, k_kv8_select<64>, k, part) : cudaLaunchKernelEx(&cfg, k_kv8_select<128>, k, part));
  }
  return NT_OK;
}
