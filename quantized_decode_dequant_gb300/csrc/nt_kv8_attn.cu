// nt_kv8_attn.cu -- attention over the paged 8-bit cache (include/nt.h,
// nt_attention_kv8).
//
// The mathematics.  For one (entry, kv head), an item, with G query heads, tiles of 128
// positions go through two products on tcgen05, kind::f8f6f4, whose A operand is the
// cache itself, copied from its page to shared memory and never decoded:
//   S^T [128 positions][6 G] = K [128][hd] . q^T        q as six e4m3 terms, each 1/16 of the one before
//   O^T [hd][8 G]            = V^T [hd][128] . P^T      the weights as eight digits
// e4m3 has four significant bits, so six terms, each the rounding of what the ones before left,
// hold q to 2^-24 and more.  A weight w in [0, 16) is a whole number, w 2^28 rounded up or down (whole_number), cut into
// eight digits of four bits: the e4m3 codes 0 to 15 are the numbers 0 to 15 times 2^-9, so a
// digit is its own code and an and and a shift make four of them.  Every product is exact; the tensor cores add
// with 2^-25 of the largest product dropped, and truncate sums, so a tile's outputs
// are taken out of tensor memory and added in registers.
//   A key's exponent multiplies its scores, a value's its weight: powers of two.  What a value's exponent lies below the largest of
// a product its weight loses in bits, so a product takes pages whose values' exponents are at most 7 apart, and a tile
// with others several products, in each of which the other pages' weights are zero.  In these products, and where a tile's values are
// larger than those of a tile before, low weights may count as much as the head's largest: they are brought up to 1.  The weights are
// 2^(score - m), m the head's largest score of the first tile, moved only where a later one passes it by
// 2^3.9.  log2(e) / sqrt(hd) is multiplied into q, so that what brings a score to the exponent is a power of two
// and the maximum and the weights see the same number however large it is.
//
// Two forms, chosen on the host (kv8_launch_attn).  Where there are few items of a small capacity, a thread-block
// cluster per item, whose CTAs share out its tiles and merge their partial results through distributed shared memory.
// Else the tiles of all items in a row go evenly to the CTAs, two per SM; an item that is cut leaves partial results for a
// second launch.  In a CTA one warp copies, one starts products, four have a position (then a dimension) per thread.
//
// What bounds it: memory while it streams.  1 sequence of 131077 positions, 64/8 heads of 128, 268 MB: 48.5 us, of which 43
// at 6.1 TB/s, the start 2, the second launch 3; 56 ragged ones, 32/8, 520 MB: 91.2; 1 with 128/8 heads: 52.2 (instructions:
// a tile takes a CTA 1800 cycles with 8 heads a kv head where it comes out of L2, 1500 with 4).  1 of 4161: 8.0 us, a chain of length, page, tile
// and q (3900 cycles to the first scores), then the cluster's merge.
#include "nt_kv8.cuh"

namespace nt {

constexpr int kKv8Batch = 512;          // entries of a launch: their first tiles are kept in shared memory
constexpr int kKv8MaxCtas = 304;        // two per SM; the workspace holds two partial results of each
constexpr int kKv8Tile = 128;
constexpr int kKv8MaxCluster = 16;
// Exponents of the values of a product: at most so far apart; largest ones of a tile: at most so far above a tile's before, else the
// tile goes the rare path.  (131077 positions, 64/8 heads, us, exponents within +-2 of their own as a model's vary: apart by 4, pages of 64 65
// and of 16 142; by 7 48.6 and 49.9, as with like ones.  All tiles on the rare path, half of the pages 2^10 larger: 148 and 203.)
constexpr int kKv8Apart = 7, kKv8Above = 4;

struct Kv8AttnArgs {
  int32_t layer, n, G, k;
  int32_t seq0;                         // sequence of entry 0 where none are listed
  const int32_t* seq;
  const int32_t* ctx;
  const int32_t* pages;
  const float* q;
  int64_t q_stride;
  float* out;
  int64_t out_stride;
  float scale;                          // log2(e) / sqrt(hd)
  float* part;                          // [CTA][2] partial results: of an item begun before this CTA, of one that goes on behind it
  int2* open;                           // [CTA]: the latter's item (-1: none) and the number of CTAs that work on it
};

// Partial result of one item: o [HB][HD], then (reference m, sum l) per head.
constexpr int kv8_part_floats(int hd, int hb) { return hb * hd + 2 * hb; }

size_t kv8_attn_ws_bytes(int hd) {
  return size_t(kKv8MaxCtas) * (2 * kv8_part_floats(hd, kKv8MaxGroup) * 4 + 8);
}

template <int HD, int HB>
struct Kv8AttnCfg {
  static constexpr int kThreads = 192;                              // four warps of the softmax, one that copies, one that starts products
  static constexpr int kTerms = 6, kDigits = 8;
  static constexpr int NS = (kTerms * HB + 15) / 16 * 16, NP = kDigits * HB;
  // ring: a tile's K, then its V, a slot each, so that K's is free again with the scores; the pages' exponents and the number
  // of positions in a ring of their own, by tile.  (As many as two CTAs an SM have room for; 131077 positions with whole tiles
  // a slot: 57.8 us, half ones 54.6, all else equal.)
  static constexpr int H = HD == 128 ? (HB <= 4 ? 6 : HB == 8 ? 5 : 4) : (HB <= 8 ? 10 : 8), E = H / 2 + 1;
  static constexpr int kSlot = kKv8Tile * HD;
  static constexpr int kPart = kv8_part_floats(HD, HB);
  static_assert(kPart * 4 <= H * kSlot, "a partial result fits the ring");
  // P^T: blocks of 8 positions by 16 rows, the digits of two heads, which a thread stores as 16 bytes; 8 positions further kPStep
  static constexpr int kPStep = NP * 8;
  // shared memory (V's rows 64 to 127 with 64 dimensions, which nobody looks at, reach 1 KB behind it)
  static constexpr int kExps = H * kSlot;
  static constexpr int kQ = kExps + E * 8 * 16;
  static constexpr int kP = kQ + NS * HD;
  static constexpr int kRed = kP + 16 * kPStep;                      // [4][HB] of the warps, twice: maxima, sums; [2][HB] scales of q
  static constexpr int kTops = kRed + 10 * HB * 4;                   // [2][4][HB] maxima over the positions of a product
  static constexpr int kLows = kTops + 8 * HB * 4;                   // [4] of each warp, see vlow
  static constexpr int kPrefix = kLows + 16;
  static constexpr int kEntry = kPrefix + (kKv8Batch + 4) * 4;
  static constexpr int kSums = kEntry + kKv8Batch * 8;
  static constexpr int kInfo = kSums + 32;                          // [E]: positions of the tile, and kLacks: behind them a page is not there
  static constexpr int kLacks = 1 << 16;
  static constexpr int kBars = (kInfo + 4 * E + 7) / 8 * 8;         // full [H], empty [H], scores, taken, weights, outputs
  static constexpr int kTmem = kBars + 8 * (2 * H + 4);
  static constexpr int kSegs = kTmem + 4;                           // items whose q is there
  static constexpr int kMore = kTmem + 8;                           // another product of the same tile's values comes behind this one
  static constexpr int kSmem = kTmem + 16;
  static_assert(kSmem <= 113 * 1024, "two CTAs an SM");
  // tensor memory: scores, outputs (twice, so that a tile's can be taken while the next one's are formed, gained nothing)
  static constexpr int kColS = 0, kColO = NS, kUsed = NS + NP, kCols = kUsed <= 32 ? 32 : kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : 256;
  static_assert(kUsed <= 256, "tensor memory of two CTAs");
};

// ------------------------------------------------------------ small pieces --

__device__ __forceinline__ float kv8_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// An operand without swizzle: blocks of 8 rows by 16 bytes; 16 bytes of k further `kstep` bytes, 8 rows further `rstep`.
__device__ __forceinline__ uint64_t kv8_desc(uint32_t a, uint32_t kstep, uint32_t rstep) {
  return uint64_t((a & 0x3ffffu) >> 4) | uint64_t(kstep >> 4) << 16 | uint64_t(rstep >> 4) << 32 | uint64_t(1) << 46;
}
__device__ __forceinline__ void kv8_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
      : "memory");
}
// this lane's row, 16 columns; awaited by kv8_tc_wait
__device__ __forceinline__ void kv8_tc_ld16(uint32_t a, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a));
}
// The loads before have arrived: n registers of theirs are named so that no use moves above.
template <int N>
__device__ __forceinline__ void kv8_tc_wait(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; i++) asm volatile("" : "+r"(r[i]));
}
// (by a whole warp, the same for all of it)
__device__ __forceinline__ bool kv8_bar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, done);
}
// Barrier of the four softmax warps; whether any of their threads says so.
__device__ __forceinline__ bool kv8_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(p))
      : "memory");
  return r;
}

// N values of every lane joined over the warp by f, value by value: halves of them are exchanged while there are several, so that it takes
// N + log2(32 / N) - 1 exchanges; lane l is left with value kv8_joined<N>(l).
template <int N, class F>
__device__ __forceinline__ float kv8_join(float (&x)[N], F f) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = N, o = 16; n > 1; n /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n / 2; i++) {
      const float got = __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + n / 2], o);
      x[i] = f(up ? x[i + n / 2] : x[i], got);
    }
  }
  float y = x[0];
#pragma unroll
  for (int o = 16 / N; o; o /= 2) y = f(y, __shfl_xor_sync(0xffffffffu, y, o));
  return y;
}
template <int N>
__device__ __forceinline__ int kv8_joined(int lane) { return lane / (32 / N); }

// Where a CTA is in the row of all tiles: tile ti of nt of kv head g of entry e.
struct Kv8At {
  int e, g, ti, nt;
};

// ------------------------------------------------------------ the kernel --

// CL: block (rank, item) of a cluster per item.
template <int HD, int HB, bool CL>
__global__ void __launch_bounds__(Kv8AttnCfg<HD, HB>::kThreads, 2) k_kv8_attn(Kv4 c, Kv8AttnArgs a) {
  using Cfg = Kv8AttnCfg<HD, HB>;
  constexpr int H = Cfg::H, E = Cfg::E, NT = Cfg::kThreads;
  extern __shared__ __align__(128) uint8_t kv8_sm[];
  uint8_t* sm = kv8_sm;
  const uint32_t smu = kv4_smem(sm);
  int* prefix = reinterpret_cast<int*>(sm + Cfg::kPrefix);
  int2* entry = reinterpret_cast<int2*>(sm + Cfg::kEntry);
  volatile int* info = reinterpret_cast<volatile int*>(sm + Cfg::kInfo);
  volatile int* segs_ready = reinterpret_cast<volatile int*>(sm + Cfg::kSegs);
  volatile int* more = reinterpret_cast<volatile int*>(sm + Cfg::kMore);
  const volatile uint32_t* tensor_memory = reinterpret_cast<const volatile uint32_t*>(sm + Cfg::kTmem);
  const uint32_t full = smu + Cfg::kBars, empty = full + 8 * H, bar_s = empty + 8 * H, bar_taken = bar_s + 8,
                 bar_p = bar_taken + 8, bar_o = bar_p + 8;
  const int t = threadIdx.x, warp = __shfl_sync(0xffffffffu, t >> 5, 0), lane = t & 31, n = a.n, P = c.page_len, lg = 31 - __clz(P);

  if (t == 0) {
    for (int i = 0; i < H; i++) {
      kv4_bar_init(full + 8 * i);
      kv4_bar_init(empty + 8 * i);
    }
    kv4_bar_init(bar_s);
    kv4_bar_init(bar_taken, 4);
    kv4_bar_init(bar_p, 4);
    kv4_bar_init(bar_o);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    *segs_ready = *more = 0;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (tensor memory only now: a kernel that this one waits for could want it on this SM; and the right to take it goes on at
  // once: the other CTA of the SM waits for it)
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smu + Cfg::kTmem), "n"(Cfg::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // ---- first tiles of all entries
  auto tiles = [&](int len) {   // of an item whose entry sees len positions
    uint32_t x = uint32_t(len);                        // (at most 2^31 - 256)
    if (a.k) x = min((x + P - 1) >> lg, uint32_t(a.k)) << lg;
    return int((x + kKv8Tile - 1) / kKv8Tile);
  };
  int2 only = make_int2(-1, 0);                        // CL: the item's entry
  int total = 0;
  if (CL) {
    uint32_t bad;
    only = kv8_entry(c, a.seq, a.ctx, a.seq0, int(blockIdx.y) / c.n_kv, &bad);
    if (bad && blockIdx.x == 0 && t == 0) kv4_flag(c, bad);
    total = tiles(only.y);
    kv4_tc_before();
    __syncthreads();
    kv4_tc_after();
  } else {
    int* sums = reinterpret_cast<int*>(sm + Cfg::kSums);
    int run = 0;
    for (int e0 = 0; e0 < n; e0 += NT) {
      const int e = e0 + t;
      int mine = 0;
      if (e < n) {
        uint32_t bad;
        const int2 sl = kv8_entry(c, a.seq, a.ctx, a.seq0, e, &bad);
        if (bad && blockIdx.x == 0) kv4_flag(c, bad);
        entry[e] = sl;
        mine = tiles(sl.y) * c.n_kv;
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
#pragma unroll
      for (int w = 0; w < NT / 32; w++) {
        const int y = sums[w];
        if (w < warp) before += y;
        all += y;
      }
      if (e < n) prefix[e] = run + before + x - mine;
      run += all;
      __syncthreads();
    }
    if (t == 0) prefix[n] = run;
    kv4_tc_before();
    __syncthreads();
    kv4_tc_after();
  }
  const uint32_t tmem = *tensor_memory;
  asm volatile("griddepcontrol.launch_dependents;");
  if (!CL) total = prefix[n];
  auto seen = [&](int e) { return CL ? only : entry[e]; };
  int share = (total + int(gridDim.x) - 1) / int(gridDim.x);
  if (share < 1) share = 1;
  const int c0 = int(blockIdx.x) * share < total ? int(blockIdx.x) * share : total, c1 = c0 + share < total ? c0 + share : total;
  float* part0 = a.part + int64_t(blockIdx.x) * 2 * Cfg::kPart;

  auto locate = [&](int x, Kv8At& at) {
    if (CL) {
      at = Kv8At{int(blockIdx.y) / c.n_kv, int(blockIdx.y) % c.n_kv, x, total};
      return;
    }
    int lo = 0, hi = n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= x) lo = mid; else hi = mid;
    }
    at.e = lo;
    at.nt = tiles(entry[lo].y);
    const int r = x - prefix[lo];
    at.g = int(uint32_t(r) / uint32_t(at.nt));
    at.ti = r - at.g * at.nt;
  };
  auto segment = [&](int x, const Kv8At& at) { return at.nt - at.ti < c1 - x ? at.nt - at.ti : c1 - x; };   // tiles up to the item's or the CTA's end

  if (warp == 4) {
    // ---- copies.  Lane y knows the page at place first + y of the item's list; the next 32 are looked up a batch ahead.
    const Kv8Page L(c);
    const uint8_t* layer_pool = c.pool + int64_t(a.layer) * c.n_pages * c.page_bytes();
    const int per = kKv8Tile >> lg, codes = P * HD;
    int no = 0, begun = 0;                             // tiles; slots filled
    bool dead = false;
    for (int x = c0; x < c1 && !dead;) {
      Kv8At at;
      locate(x, at);
      const int count = segment(x, at), len = seen(at.e).y;
      const int m = int((uint32_t(len) + P - 1) >> lg), listed = a.k && a.k < m ? a.k : m;
      const int32_t* row = c.table + int64_t(seen(at.e).x) * c.max_pages;
      const int32_t* list = a.k ? a.pages + (int64_t(at.e) * c.n_kv + at.g) * a.k : nullptr;
      const int end = (at.ti + count) * per < listed ? (at.ti + count) * per : listed;
      // the page at place i of the list; -1: none there, -2: the list has ended; *last: it is the sequence's last page
      auto look = [&](int i, bool* last) -> int {
        *last = false;
        if (i >= end) return -2;
        int j = i;
        if (list) {
          j = list[i];
          const int before = i ? list[i - 1] : -1;
          if (j < 0) return -2;
          if (j >= m || j <= before || (i && before < 0)) { kv4_flag(c, NT_KV4_BAD_PAGE); return -1; }
        }
        *last = j == m - 1;
        const int page = row[j];
        if (page < 0 || page >= c.n_pages) { kv4_flag(c, NT_KV4_BAD_PAGE); return -1; }
        return page;
      };
      bool last, next_last;
      int first = at.ti * per, page = look(first + lane, &last), next = look(first + 32 + lane, &next_last);
      for (int i = 0; i < count; i++, no++) {
        const int at_list = (at.ti + i) * per;
        if (at_list - first >= 32) {
          first += 32;
          page = next;
          last = next_last;
          next = look(first + 32 + lane, &next_last);
        }
        const int y = at_list - first + lane % 8;
        const int mine = __shfl_sync(0xffffffffu, page, y & 31);
        const bool is_last = __shfl_sync(0xffffffffu, int(last), y & 31);
        // what lies behind a page that is not there is not looked at either
        const uint32_t lacking = __ballot_sync(0xffffffffu, lane < per && mine == -1);
        const bool live = lane % 8 < per && mine >= 0 && (lacking == 0u || lane % 8 < __ffs(lacking) - 1);
        const int have = __popc(__ballot_sync(0xffffffffu, lane < 8 && live));
        const bool ends = __any_sync(0xffffffffu, live && is_last), nothing = !have;
        const uint8_t* from = layer_pool + (live ? mine : 0) * c.page_bytes();
#pragma unroll
        for (int v = 0; v < 2; v++) {                  // K, V
          const int fill = 2 * no + v, slot = fill % H;
          if (fill >= H && !__all_sync(0xffffffffu, kv4_bar_wait(empty + 8 * slot, uint32_t(fill / H - 1) & 1u))) { dead = true; break; }
          const uint32_t bar = full + 8 * slot;
          if (lane == 0) {
            if (v == 0) info[no % E] = (have * P - (ends ? m * P - len : 0)) | (lacking ? Cfg::kLacks : 0);
            if (nothing) kv4_bar_arrive(bar);
            else kv4_bar_expect(bar, uint32_t(have) * uint32_t(codes + (v ? 0 : 16)));
          }
          __syncwarp();
          if (!nothing && live && lane < (v ? 8 : 16)) {
            const int z = lane % 8;
            if (lane < 8) kv4_copy(smu + slot * Cfg::kSlot + z * codes, from + (v ? L.v(at.g) : L.k(at.g)), codes, bar);
            else kv4_copy(smu + Cfg::kExps + (no % E * 8 + z) * 16, from + L.exps(at.g), 16, bar);
          }
          begun = fill + 1;
        }
        if (dead) break;
      }
      x += count;
    }
    if (dead) {   // copies in flight land before the shared memory is given up
      if (lane == 0) kv4_flag(c, NT_KV4_TIMEOUT);
      for (int i = begun < H ? 0 : begun - H; i < begun; i++) kv4_bar_wait(full + 8 * (i % H), uint32_t(i / H) & 1u);
    }
  } else if (warp == 5) {
    // ---- products: scores of tile ns as soon as it and q are there and the scores before are taken, outputs of
    // tile np as soon as its weights are there, whichever comes first
    constexpr uint32_t kIdesc = 1u << 4 | uint32_t(kKv8Tile / 16) << 24;   // fp32 += e4m3 e4m3, 128 rows
    constexpr uint32_t kIdescS = kIdesc | uint32_t(Cfg::NS / 8) << 17, kIdescO = kIdesc | uint32_t(Cfg::NP / 8) << 17 | 1u << 16;   // P^T: rows side by side
    const int all = c1 - c0;
    int ns = 0, np = 0, weighed = 0, segs = 0, left = 0, idle = 0;   // left: tiles of the segment without scores
    bool has_k = false, has_v = false;                 // tile ns has its K, tile np its V
    while (np < all) {
      bool moved = false;
      if (ns < all && ns - np < E - 1) {
        const int slot = 2 * ns % H;
        bool ok = true;
        if (left == 0) {
          ok = __all_sync(0xffffffffu, *segs_ready > segs);   // (a count: items without a live tile may pass several at a time)
          if (ok) {
            Kv8At at;
            locate(c0 + ns, at);
            left = segment(c0 + ns, at);
            segs++;
          }
        }
        if (!has_k) has_k = kv8_bar_test(full + 8 * slot, uint32_t(2 * ns / H) & 1u);
        if (ok && has_k && (ns == 0 || kv8_bar_test(bar_taken, uint32_t(ns - 1) & 1u))) {
          if (info[ns % E] & (Cfg::kLacks - 1)) {
            kv4_tc_after();
            if (kv4_elect()) {
              const uint32_t k0 = smu + slot * Cfg::kSlot, q0 = smu + Cfg::kQ;
#pragma unroll
              for (int kk = 0; kk < HD / 32; kk++)
                kv8_mma(tmem + Cfg::kColS, kv8_desc(k0 + kk * 256, 128, 8 * HD), kv8_desc(q0 + kk * 256, 128, 8 * HD), kIdescS, kk > 0);
              kv4_tc_commit(bar_s);
              kv4_tc_commit(empty + 8 * slot);
            }
          } else if (lane == 0) {                      // nothing to multiply: the tile goes the same way
            kv4_bar_arrive(bar_s);
            kv4_bar_arrive(empty + 8 * slot);
          }
          __syncwarp();
          has_k = false;
          ns++;
          left--;
          moved = true;
        }
      }
      if (np < ns) {
        const int fill = 2 * np + 1, slot = fill % H;
        if (!has_v) has_v = kv8_bar_test(full + 8 * slot, uint32_t(fill / H) & 1u);
        if (has_v) {
          if (!(info[np % E] & (Cfg::kLacks - 1))) {                     // free once the softmax warps have seen that there is nothing
            if (ns > np + 1 || kv8_bar_test(bar_taken, uint32_t(np) & 1u)) {
              if (lane == 0) kv4_bar_arrive(empty + 8 * slot);
              __syncwarp();
              has_v = false;
              np++;
              moved = true;
            }
          } else if (kv8_bar_test(bar_p, uint32_t(weighed) & 1u)) {
            const bool last = !*more;
            kv4_tc_after();
            if (kv4_elect()) {
              const uint32_t v0 = smu + slot * Cfg::kSlot, p0 = smu + Cfg::kP;
#pragma unroll
              for (int kk = 0; kk < kKv8Tile / 32; kk++)
                kv8_mma(tmem + Cfg::kColO, kv8_desc(v0 + kk * 32 * HD, 16 * HD, 128),
                        kv8_desc(p0 + kk * 4 * Cfg::kPStep, Cfg::kPStep, 128), kIdescO, kk > 0);
              kv4_tc_commit(bar_o);
              if (last) kv4_tc_commit(empty + 8 * slot);
            }
            __syncwarp();
            weighed++;
            if (last) {
              has_v = false;
              np++;
            }
            moved = true;
          }
        }
      }
      idle = moved ? 0 : idle + 1;
      if (idle > (1 << 24)) {
        if (lane == 0) kv4_flag(c, NT_KV4_TIMEOUT);
        break;
      }
    }
  } else {
    // ---- softmax: thread t has position t of a tile, and dimension t of the outputs
    const uint32_t mine = uint32_t(32 * warp) << 16;   // this warp's rows of tensor memory
    float* red = reinterpret_cast<float*>(sm + Cfg::kRed);
    uint8_t* my_p = sm + Cfg::kP + (t >> 3) * Cfg::kPStep + (t & 7) * 16;
    float O[HB], l[HB], mref[HB], css[HB];
    uint32_t ps = 0, po = 0;
    int no = 0, segs = 0;                              // tiles; items whose q was prepared
    bool dead = false;
    // outputs of the last tile with scores: none under way, under way, there; their scale
    int pending = 0;
    float out_scale = 0.f;
    // of the item's tiles so far: the smallest of their largest value exponents
    volatile int* vlow = reinterpret_cast<volatile int*>(sm + Cfg::kLows) + warp;
    auto await = [&]() -> bool {                       // false: they never came
      if (pending != 1) return true;
      pending = 2;
      const bool ok = __all_sync(0xffffffffu, kv4_bar_wait(bar_o, po));
      po ^= 1u;
      kv4_tc_after();
      return ok;
    };
    constexpr int kTake = HB < 4 ? HB : 4;             // heads taken together
    const uint64_t k16 = kv8_pack(16.f, 16.f), k65536 = kv8_pack(65536.f, 65536.f);
    auto output = [&](const uint32_t* r) {             // out of the sums of a head's digits 0, 2, 4, 6, 1, 3, 5, 7
      auto two = [&](int i) { return kv8_pack(__uint_as_float(r[i]), __uint_as_float(r[i + 1])); };
      const float2 v = kv8_unpack(kv8_fma2(kv8_fma2(two(6), k16, two(2)), k65536, kv8_fma2(two(4), k16, two(0))));
      return fmaf(v.y, 256.f, v.x);
    };
    auto take = [&]() {                                // adds them to the sums
      if (pending != 2) return;
      pending = 0;
      const uint32_t from = tmem + mine + Cfg::kColO;
      if (HD == 128 || warp < 2) {
#pragma unroll
        for (int b = 0; b < HB / kTake; b++) {
          uint32_t r[8 * kTake];
#pragma unroll
          for (int y = 0; y < kTake / 2; y++) kv8_tc_ld16(from + 8 * kTake * b + 16 * y, r + 16 * y);
          kv8_tc_wait(r);
#pragma unroll
          for (int h = 0; h < kTake; h++) O[kTake * b + h] = fmaf(output(r + 8 * h), out_scale, O[kTake * b + h]);
        }
      }
      kv4_tc_before();
    };

    // The q of the item at `at` into shared memory, scaled so that its largest element is in [2^7, 2^8), in six terms; a warp takes every fourth
    // row.  It is done before the item before it is finished with, once that one's scores are all there.
    float* scales = red + 8 * HB;
    auto prepare = [&](const Kv8At& at, int odd) {
      constexpr int V = HD / 32;
      constexpr int kMine = (HB + 3) / 4;            // rows of a warp: all on the way together
      float z[kMine][V];
#pragma unroll
      for (int j = 0; j < kMine; j++) {
        const int h = warp + 4 * j;
        const float* qb = a.q + int64_t(at.e) * a.q_stride + (int64_t(at.g) * a.G + h) * HD + V * lane;
#pragma unroll
        for (int i = 0; i < V; i++) z[j][i] = 0.f;
        if (h < a.G) {
          if (V == 4) {
            const float4 w = *reinterpret_cast<const float4*>(qb);
            z[j][0] = w.x; z[j][1] = w.y; z[j][2 % V] = w.z; z[j][3 % V] = w.w;
          } else {
            const float2 w = *reinterpret_cast<const float2*>(qb);
            z[j][0] = w.x; z[j][1] = w.y;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kMine; j++) {
        const int h = warp + 4 * j;
        if (h >= HB) break;
        float (&y)[V] = z[j], top = 0.f;
#pragma unroll
        for (int i = 0; i < V; i++) {
          y[i] *= a.scale;
          if (!(fabsf(y[i]) < INFINITY)) y[i] = NAN;
          top = fmaxf(top, fabsf(y[i]));             // (a NaN is passed over)
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        int ex = int(__float_as_uint(top) >> 23);
        ex = ex < 14 ? 14 : ex;                      // (zeros and values below 2^-113)
        const float up = __uint_as_float(uint32_t(261 - ex) << 23);                  // 2^(134 - ex)
        if (lane == 0) scales[odd * HB + h] = __uint_as_float(uint32_t(ex - 7) << 23);             // 2^(ex - 134)
        uint8_t* to = sm + Cfg::kQ + (V * lane >> 4) * 128 + (V * lane & 15);
#pragma unroll
        for (int i = 0; i < V; i++) y[i] *= up;
#pragma unroll
        for (int k = 0; k < Cfg::kTerms; k++) {
          const int row = k * HB + h;
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const uint32_t w = kv8_code2(y[i], y[i + 1]);
            *reinterpret_cast<uint16_t*>(to + (row >> 3) * 8 * HD + (row & 7) * 16 + i) = uint16_t(w);
            const float2 f = kv8_value2(w);
            y[i] = (y[i] - f.x) * 16.f;
            y[i + 1] = (y[i + 1] - f.y) * 16.f;
          }
        }
      }
      if constexpr (Cfg::NS > Cfg::kTerms * HB)      // rows of no head
        for (int i = t; i < (Cfg::NS - Cfg::kTerms * HB) * HD / 16; i += 128) {
          const int row = Cfg::kTerms * HB + i / (HD / 16);
          *reinterpret_cast<uint4*>(sm + Cfg::kQ + (row >> 3) * 8 * HD + i % (HD / 16) * 128 + (row & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      kv8_any(false);
      if (t == 0) {
        __threadfence_block();
        *segs_ready = ++segs;
      }
    };
    Kv8At at, next;
    if (c0 < c1) {
      locate(c0, next);
      prepare(next, 0);
    }
    int odd = 0;
#pragma unroll 1
    for (int x = c0; x < c1; odd ^= 1) {
      at = next;
      const int count = segment(x, at);
      bool poison = dead;
      auto cs = [&](int h) { return HB == 16 && HD == 128 ? scales[odd * HB + h] : css[h]; };   // (16 more registers are not there; with 64 dimensions they are)
#pragma unroll
      for (int h = 0; h < HB; h++) {
        css[h] = scales[odd * HB + h];
        O[h] = l[h] = 0.f;
        mref[h] = -3e38f;
      }
      if (lane == 0) *vlow = 127;
      uint32_t turn = uint32_t((at.ti - 1) * kKv8Tile + t) * 0x9e3779b9u;   // of position t: of the golden ratio, without whole ones
      __syncwarp();
#pragma unroll 1
      for (int i = 0; i < count; i++, no++) {
        turn += kKv8Tile * 0x9e3779b9u;
        if (dead) continue;
        // (not K's own barrier: its slot may have been filled again by now)
        bool fail = !__all_sync(0xffffffffu, kv4_bar_wait(bar_s, ps));
        ps ^= 1u;
        const int word = info[no % E], live = word & (Cfg::kLacks - 1);
        if (word & Cfg::kLacks) poison = true;
        if (live == 0 || fail) {
          if (kv8_any(fail)) dead = kv8_any(fail) && kv8_any(fail);     // (as many barriers as a tile with scores has)
          poison = poison || dead;
          __syncwarp();
          if (lane == 0) kv4_bar_arrive(bar_taken);
          continue;
        }
        kv4_tc_after();
        if (live < kKv8Tile) {   // values behind the end: zeros, whatever the page holds there
          const int vfill = 2 * no + 1;
          fail = !__all_sync(0xffffffffu, kv4_bar_wait(full + 8 * (vfill % H), uint32_t(vfill / H) & 1u)) || fail;
          uint8_t* v = sm + vfill % H * Cfg::kSlot;
          if (t < HD)
            for (int ch = live >> 4; ch < 8; ch++) {
              uint4* at16 = reinterpret_cast<uint4*>(v + kv8_v_at(HD, ch, t));
              uint4 w = make_uint4(0u, 0u, 0u, 0u);
              const int keep = live - 16 * ch;         // bytes that stay
              if (keep > 0) {
                w = *at16;
                auto cut = [&](uint32_t z, int b) { return keep >= b + 4 ? z : keep <= b ? 0u : z & ((1u << (8 * (keep - b))) - 1u); };
                w = make_uint4(cut(w.x, 0), cut(w.y, 4), cut(w.z, 8), cut(w.w, 12));
              }
              *at16 = w;
            }
        }
        // ---- scores; while they come, the exponents of the tile's pages: this position's key's and value's, the largest value's
        float s[HB], fk, fv;
        int vmax;
        {
          constexpr int kParts = HB == 16 ? 2 : 1, kCols = Cfg::NS / kParts, kT = Cfg::kTerms / kParts;   // with 16 heads three terms at a time
          const int8_t* exps = reinterpret_cast<const int8_t*>(sm + Cfg::kExps + no % E * 8 * 16);
#pragma unroll
          for (int b = kParts - 1; b >= 0; b--) {
            uint32_t r[kCols];
#pragma unroll
            for (int y = 0; y < kCols / 16; y++) kv8_tc_ld16(tmem + mine + Cfg::kColS + b * kCols + 16 * y, r + 16 * y);
            if (b == kParts - 1) {
              const int of = t < live ? t >> lg : 0, ek = exps[16 * of], ev = exps[16 * of + 1], low = *vlow;
              vmax = __reduce_max_sync(0xffffffffu, (lane & 7) << lg < live ? int(exps[16 * (lane & 7) + 1]) : -128);
              fk = kv8_exp2i(ek);
              fv = ev < vmax - kKv8Apart || vmax > low + kKv8Above ? 0.f : kv8_exp2i(28 + ev - vmax);
              *vlow = min(vmax, low);
            }
            kv8_tc_wait(r);
            if (b == 0) {
              kv4_tc_before();
              __syncwarp();
              if (lane == 0) kv4_bar_arrive(bar_taken);
            }
            const uint64_t k16th = kv8_pack(1.f / 16.f, 1.f / 16.f);
#pragma unroll
            for (int h = 0; h < HB; h += 2) {
              auto two = [&](int k) { return kv8_pack(__uint_as_float(r[k * HB + h]), __uint_as_float(r[k * HB + h + 1])); };
              uint64_t z = two(kT - 1);
              if (b < kParts - 1) z = kv8_fma2(kv8_pack(s[h], s[h + 1]), k16th, z);
#pragma unroll
              for (int k = kT - 2; k >= 0; k--) z = kv8_fma2(z, k16th, two(k));
              const float2 y = kv8_unpack(z);
              s[h] = y.x;
              s[h + 1] = y.y;
            }
          }
        }
#pragma unroll
        for (int h = 0; h < HB; h++) s[h] = t < live ? s[h] * fk : -INFINITY;
        // ---- weights
        float p[HB], most;
        auto weights = [&]() {
          most = 0.f;
#pragma unroll
          for (int h = 0; h < HB; h++) {
            p[h] = kv8_ex2(fmaf(s[h], cs(h), -mref[h]));
            most = fmaxf(most, p[h]);
          }
        };
        auto digits = [&](int h, uint32_t u0, uint32_t u1) {   // of two heads' weights times 2^28
          *reinterpret_cast<uint4*>(my_p + h * 64) =
              make_uint4(u0 & 0x0f0f0f0fu, (u0 >> 4) & 0x0f0f0f0fu, u1 & 0x0f0f0f0fu, (u1 >> 4) & 0x0f0f0f0fu);
        };
        // A weight's whole number is rounded up where its fraction lies less than a gap below the next, a gap of its position's own; they
        // are multiples of the golden ratio without their whole part, evenly spread, so that of many weights below the last digit as many
        // get one as make up their sum.  (Rounded to the nearest, all of them were lost: n 2^-29 of the largest weight.  It costs
        // nothing with heads of 128; 64/8 heads of 64, 262000 positions 54.6 -> 55.2 us.)
        auto gap_of = [&]() { return __uint_as_float(turn >> 9 | 0x3f800000u) - 1.f; };
        auto whole_number = [&](float w, float gap) { return __float2uint_rz(__fmaf_rz(w, fv, gap)); };
        auto multiply = [&]() {                        // the product with these digits
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          kv4_tc_before();
          __syncwarp();
          if (lane == 0) kv4_bar_arrive(bar_p);
          out_scale = kv8_exp2i(vmax - 19);            // digits are 2^-9 of themselves, weights 2^28
          pending = 1;
        };
        weights();
        if (kv8_any(!(most <= 15.f) || fail || fv == 0.f)) {
          // A weight may have passed 2^3.9 (at first all are infinite): the maxima over the tile's positions.
          fail = !await() || fail;
          take();
          {
            float x[HB];
#pragma unroll
            for (int h = 0; h < HB; h++) x[h] = s[h];
            const float top = kv8_join(x, [](float u, float v) { return fmaxf(u, v); });
            if (lane % (32 / HB) == 0) red[warp * HB + kv8_joined<HB>(lane)] = top;
          }
          const bool apart = kv8_any(fail || fv == 0.f);
          dead = apart && kv8_any(fail);
#pragma unroll
          for (int h = 0; h < HB; h++) {
            const float top = fmaxf(fmaxf(red[h], red[HB + h]), fmaxf(red[2 * HB + h], red[3 * HB + h])) * cs(h);
            const float to = top - mref[h] > 3.f ? top : mref[h], f = kv8_ex2(mref[h] - to);
            mref[h] = to;
            l[h] *= f;
            O[h] *= f;
          }
          if (dead) {
            poison = true;
            continue;
          }
          if (apart) {
            // Values too small for a product with the tile's largest, or larger than those of the tiles before: a product for those that go
            // together, the largest first, with the weights of a head brought up to 1 where all are lower.  (Rare: little code, few registers; the
            // arrays are in local memory.)
            float x[HB], o[HB], sum[HB];
#pragma unroll
            for (int h = 0; h < HB; h++) {
              x[h] = fmaf(s[h], cs(h), -mref[h]);
              o[h] = O[h];
              sum[h] = l[h];
            }
            const int8_t* exps = reinterpret_cast<const int8_t*>(sm + Cfg::kExps + no % E * 8 * 16);
            const int ev = exps[16 * (t < live ? t >> lg : 0) + 1], page = exps[16 * ((lane & 7) << lg < live ? lane & 7 : 0) + 1];
            float* tops = reinterpret_cast<float*>(sm + Cfg::kTops);
#pragma unroll 1
            for (int next = vmax, above = 128, other = 4 * HB; next > -129; tops += other, other = -other) {
              vmax = next;
              const int least = vmax - kKv8Apart;
              const bool in = ev < above && ev >= least;
              fv = in ? kv8_exp2i(28 + ev - vmax) : 0.f;
              above = least;
              next = __reduce_max_sync(0xffffffffu, page < least ? page : -129);
              const float gap = gap_of();
              float up = 0.f;                            // of head `lane`
              int largest = 0;
              auto ordered = [](int y) { return y ^ (y >> 31 & 0x7fffffff); };   // numbers' bits in the order of whole numbers
#pragma unroll 2
              for (int h = 0; h < HB; h++) {
                const int y = __reduce_max_sync(0xffffffffu, ordered(__float_as_int(in ? x[h] : -INFINITY)));
                if (lane == h) largest = y;
              }
              if (lane < HB) tops[warp * HB + lane] = __int_as_float(ordered(largest));
              kv8_any(false);
              if (lane < HB) {
                const float y = fmaxf(fmaxf(tops[lane], tops[HB + lane]), fmaxf(tops[2 * HB + lane], tops[3 * HB + lane]));
                up = fminf(fmaxf(floorf(-y), 0.f), 126.f);
              }
              __syncwarp();
#pragma unroll 2
              for (int h = 0; h < HB; h += 2) {
                uint32_t u[2];
#pragma unroll
                for (int y = 0; y < 2; y++) {
                  const float z = __shfl_sync(0xffffffffu, up, h + y), w = in ? kv8_ex2(x[h + y] + z) : 0.f;
                  sum[h + y] = fmaf(w, kv8_exp2i(-int(z)), sum[h + y]);
                  u[y] = whole_number(w, gap);
                }
                digits(h, u[0], u[1]);
              }
              if (t == 0) *more = next > -129;
              multiply();
              if (!await()) poison = true;
              pending = 0;
#pragma unroll 2
              for (int h = 0; h < HB && (HD == 128 || warp < 2); h += 2) {
                uint32_t r[16];
                kv8_tc_ld16(tmem + mine + Cfg::kColO + 8 * h, r);
                kv8_tc_wait(r);
#pragma unroll
                for (int y = 0; y < 2; y++)
                  o[h + y] = fmaf(output(r + 8 * y), out_scale * kv8_exp2i(-int(__shfl_sync(0xffffffffu, up, h + y))), o[h + y]);
              }
              kv4_tc_before();
            }
            if (lane == 0 && vmax < *vlow) *vlow = vmax;
#pragma unroll
            for (int h = 0; h < HB; h++) {
              O[h] = o[h];
              l[h] = sum[h];
            }
            continue;
          }
          weights();
        }
        if (!await()) poison = true;                   // (the last product has read its weights)
        take();
        const float gap = gap_of();
#pragma unroll
        for (int h = 0; h < HB; h += 2) {
          digits(h, whole_number(p[h], gap), whole_number(p[h + 1], gap));
        }
        multiply();
#pragma unroll
        for (int h = 0; h < HB; h++) l[h] += p[h];
      }
      // ---- the segment's end, behind the next one's q
      if (x + count < c1) {
        locate(x + count, next);
        prepare(next, odd ^ 1);
      }
      if (!await() || dead) poison = true;
      take();
      float* sums = red + 4 * HB;
      {
        const float sum = kv8_join(l, [](float u, float v) { return u + v; });
        if (lane % (32 / HB) == 0) sums[warp * HB + kv8_joined<HB>(lane)] = sum;
      }
      poison = kv8_any(poison);
      const bool whole = !CL && at.ti == 0 && count == at.nt, begun = at.ti == 0;
      float* part = CL ? reinterpret_cast<float*>(sm) : part0 + (begun ? Cfg::kPart : 0);
      if (t < HB) {                                    // what row t's outputs are multiplied by
        float sum = (sums[t] + sums[HB + t]) + (sums[2 * HB + t] + sums[3 * HB + t]);
        if (poison) sum = NAN;
        red[t] = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
        if (!whole) part[HB * HD + 2 * t + 1] = sum;
      }
      if (!whole && t == 0) {
#pragma unroll
        for (int h = 0; h < HB; h++) part[HB * HD + 2 * h] = mref[h];
      }
      kv8_any(false);
      float* to = (whole ? a.out + int64_t(at.e) * a.out_stride + int64_t(at.g) * a.G * HD : part) + t;
#pragma unroll
      for (int h = 0; h < HB; h++)
        if (h < a.G && t < HD) to[h * HD] = O[h] * red[h];
      x += count;
      // the CTA's last item is open where it was begun here and goes on behind
      if (!CL && x >= c1 && t == 0)
        a.open[blockIdx.x] = begun && !whole ? make_int2(at.e * c.n_kv + at.g, (x - count + at.nt - 1) / share - int(blockIdx.x) + 1) : make_int2(-1, 0);
    }
    if (!CL) {
      if (c0 >= c1 && t == 0) a.open[blockIdx.x] = make_int2(-1, 0);
      // entries without a position: zeros, or NaN where they cannot be read
      for (int e = blockIdx.x; e < n; e += gridDim.x)
        if (entry[e].y == 0)
          for (int y = t; y < c.n_kv * a.G * HD; y += 128) a.out[int64_t(e) * a.out_stride + y] = entry[e].x < 0 ? NAN : 0.f;
    } else if (c0 >= c1) {                             // no tile of this CTA's
      float* to = reinterpret_cast<float*>(sm);
      for (int y = t; y < HB * HD; y += 128) to[y] = 0.f;
      if (t < HB) reinterpret_cast<float2*>(to + HB * HD)[t] = make_float2(-3e38f, 0.f);
    }
  }
  kv4_tc_before();
  if (CL) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  else __syncthreads();
  if (warp == 5) {
    kv4_tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(Cfg::kCols));
  }
  if (CL) {
    // ---- the item's partial results, each CTA a share of the outputs, in the ranks' order
    const int ranks = int(gridDim.x), outs = a.G * HD;
    float* out = a.out + int64_t(int(blockIdx.y) / c.n_kv) * a.out_stride + int64_t(int(blockIdx.y) % c.n_kv) * outs;
    auto there = [&](int r, uint32_t at) {             // shared memory of rank r
      uint32_t y;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"(smu + at), "r"(r));
      return y;
    };
    auto load = [](uint32_t at) {
      float y;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(y) : "r"(at));
      return y;
    };
    for (int i = int(blockIdx.x) * NT + t; i < outs; i += ranks * NT) {
      const int h = i / HD;
      float m[kKv8MaxCluster], l[kKv8MaxCluster], o[kKv8MaxCluster], top = -INFINITY;
#pragma unroll
      for (int r = 0; r < kKv8MaxCluster; r++) {
        if (r >= ranks) break;
        m[r] = load(there(r, (HB * HD + 2 * h) * 4));
        l[r] = load(there(r, (HB * HD + 2 * h + 1) * 4));
        o[r] = load(there(r, i * 4));
      }
#pragma unroll
      for (int r = 0; r < kKv8MaxCluster; r++)
        if (r < ranks) top = fmaxf(top, m[r]);
      float sum = 0.f, y = 0.f;
#pragma unroll
      for (int r = 0; r < kKv8MaxCluster; r++)
        if (r < ranks) {
          const float f = kv8_ex2(m[r] - top);
          sum = fmaf(l[r], f, sum);
          y = fmaf(o[r], f, y);
        }
      out[i] = only.x < 0 ? NAN : sum == 0.f ? 0.f : y / sum;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");   // all have read this CTA's
  }
}

// Items that were cut: block (x, y) merges rows y 8 / per .. of what CTA c began, the x-th of those that left an item open, with what the next
// ones left, in their order; `per` warps a row.
constexpr int kKv8MergeWarps = 8;
template <int HD>
__global__ void __launch_bounds__(32 * kKv8MergeWarps) k_kv8_merge(Kv4 c, Kv8AttnArgs a, int ctas, int part_floats, int rows, int per) {
  constexpr int V = HD / 32, NW = kKv8MergeWarps, NT = 32 * NW, kFew = 5;   // partial results of a warp on the way together
  __shared__ float s_o[NW][HD];
  __shared__ float2 s_ml[NW];
  __shared__ int s_count[NW];
  __shared__ int s_cta, s_item, s_members;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, h = int(blockIdx.y) * (NW / per) + warp / per, rank = warp % per;
  if (t == 0) s_cta = -1;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (int(gridDim.x) >= ctas - 1) {   // as many blocks as CTAs: no need to count
    const int2 x = __ldcg(a.open + blockIdx.x);
    if (x.x < 0) return;
    if (t == 0) { s_cta = int(blockIdx.x); s_item = x.x; s_members = x.y; }
    __syncthreads();
  } else {
    int before = 0;
    for (int i0 = 0; i0 < ctas; i0 += NT) {
      const int2 x = i0 + t < ctas ? __ldcg(a.open + i0 + t) : make_int2(-1, 0);
      const uint32_t m = __ballot_sync(0xffffffffu, x.x >= 0);
      if (lane == 0) s_count[warp] = __popc(m);
      __syncthreads();
      int mine = before;
#pragma unroll
      for (int w = 0; w < NW; w++) {
        if (w < warp) mine += s_count[w];
        before += s_count[w];
      }
      if (x.x >= 0 && mine + __popc(m & ((1u << lane) - 1u)) == int(blockIdx.x)) {
        s_cta = i0 + t;
        s_item = x.x;
        s_members = x.y;
      }
      __syncthreads();
      if (before > int(blockIdx.x)) break;
    }
  }
  if (s_cta < 0) return;
  const int members = s_members, all = a.G;
  const float* first = a.part + (int64_t(s_cta) * 2 + 1) * part_floats;    // the second of this CTA, then the first of the next ones
  float M = -INFINITY, sum = 0.f, o[V];
#pragma unroll
  for (int v = 0; v < V; v++) o[v] = 0.f;
  for (int b0 = rank; b0 < members && h < all; b0 += kFew * per) {
    float2 ml[kFew];
    float x[kFew][V];
#pragma unroll
    for (int u = 0; u < kFew; u++) {
      const int b = b0 + u * per;
      if (b >= members) break;
      const float* r = b ? first + (int64_t(b) * 2 - 1) * part_floats : first;
      ml[u] = __ldcg(reinterpret_cast<const float2*>(r + rows * HD) + h);
#pragma unroll
      for (int v = 0; v < V; v++) x[u][v] = __ldcg(r + h * HD + 32 * v + lane);
    }
#pragma unroll
    for (int u = 0; u < kFew; u++) {
      if (b0 + u * per >= members) break;
      const float to = fmaxf(M, ml[u].x), was = kv8_ex2(M - to), f = kv8_ex2(ml[u].x - to);
      M = to;
      sum = fmaf(sum, was, ml[u].y * f);
#pragma unroll
      for (int v = 0; v < V; v++) o[v] = fmaf(o[v], was, x[u][v] * f);
    }
  }
#pragma unroll
  for (int v = 0; v < V; v++) s_o[warp][32 * v + lane] = o[v];
  if (lane == 0) s_ml[warp] = make_float2(M, sum);
  __syncthreads();
  const int e = s_item / c.n_kv, g = s_item % c.n_kv;
  for (int i = t; i < NW / per * HD; i += NT) {
    const int j = i / HD, d = i % HD, row = int(blockIdx.y) * (NW / per) + j;
    if (row >= all) break;
    float top = -INFINITY, total = 0.f, y = 0.f;
    for (int w = j * per; w < (j + 1) * per; w++) top = fmaxf(top, s_ml[w].x);
    for (int w = j * per; w < (j + 1) * per; w++) {
      const float f = kv8_ex2(s_ml[w].x - top);
      total = fmaf(s_ml[w].y, f, total);
      y = fmaf(s_o[w][d], f, y);
    }
    a.out[int64_t(e) * a.out_stride + (int64_t(g) * a.G + row) * HD + d] = total == 0.f ? 0.f : y / total;
  }
}

// CTAs of a cluster, and how many such clusters of the attention kernel the GPU holds at once (0: none).
constexpr int kKv8Clusters[8] = {1, 2, 3, 4, 6, 8, 12, 16};
struct Kv8Fit {
  KernelSetup setup;
  int clusters[8] = {};
};
static void kv8_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster) {
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg = cudaLaunchConfig_t{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
}
template <int HD, int HB>
static Kv8Fit kv8_fit() {
  using Cfg = Kv8AttnCfg<HD, HB>;
  Kv8Fit f;
  f.setup = kernel_setup(k_kv8_attn<HD, HB, true>, Cfg::kSmem);
  if (f.setup.err == cudaSuccess) f.setup.err = cudaFuncSetAttribute(k_kv8_attn<HD, HB, true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  for (int i = 0; i < 8 && f.setup.err == cudaSuccess; i++) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    kv8_config(cfg, attr, dim3(unsigned(kKv8Clusters[i])), Cfg::kThreads, Cfg::kSmem, nullptr, kKv8Clusters[i]);
    cfg.numAttrs = 1;
    attr[0] = attr[1];
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, k_kv8_attn<HD, HB, true>, &cfg) == cudaSuccess) f.clusters[i] = n;
    else cudaGetLastError();   // (no such cluster: it is not taken)
  }
  return f;
}

// Most tiles of a CTA in the form with a cluster per item: as many as there are items, 7 at most, and 3 (16 query heads per kv head:
// 2) more, since the more items there are, the more tiles a CTA of the other form has, and the longer its second launch takes.  (us, that
// form and the other, heads of 128.  8/1 heads, 1 sequence of 600 positions: 6.0, 7.2; 7000, 4 tiles a CTA: 8.1, 8.3; 9000, 5: 8.8,
// 8.5.  16/2, 12000, 6: 9.6, 9.7.  64/8, 4161, 3: 7.9, 9.2; 8000, 6: 9.7, 11.9; 12000, 8: 11.3, 12.8; 16000, 11: 14.4, 13.9; 20000,
// 14: 17.1, 16.6.  32/8, 2 of 9000, 9: 13.2, 14.4; 16 of 1000, 8: 11.1, 12.1.  16/1, 6000, 3: 9.3, 9.5; 8000, 4: 10.3, 9.7; 128/8,
// 8000, 6: 12.6, 15.2.)
constexpr int kKv8ClusterShare[2] = {3, 2};

template <int HD, int HB>
static cudaError_t kv8_launch_attn(const Kv4& k, const Kv8AttnArgs& a, int64_t item_tiles, cudaStream_t s) {
  using Cfg = Kv8AttnCfg<HD, HB>;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  const int64_t items = int64_t(a.n) * k.n_kv;
  // A cluster per item where all of them fit the GPU at once and their capacity leaves no CTA too many tiles: the smallest
  // cluster such that a CTA has one tile at most, or the largest.
  const int64_t most = kKv8ClusterShare[HB == 16] + (items < 7 ? items : 7);
  static const Kv8Fit fit = kv8_fit<HD, HB>();
  if (fit.setup.err != cudaSuccess) return fit.setup.err;
  int cluster = 0;
  for (int i = 0; i < 8; i++) {
    if (fit.clusters[i] < items || item_tiles > kKv8Clusters[i] * most) continue;
    cluster = kKv8Clusters[i];
    if (item_tiles <= cluster) break;
  }
  if (cluster) {
    kv8_config(cfg, attr, dim3(unsigned(cluster), unsigned(items)), Cfg::kThreads, Cfg::kSmem, s, cluster);
    return cudaLaunchKernelEx(&cfg, k_kv8_attn<HD, HB, true>, k, a);
  }
  static const KernelSetup setup = kernel_setup(k_kv8_attn<HD, HB, false>, Cfg::kSmem);
  if (setup.err != cudaSuccess) return setup.err;
  int64_t ctas = 2 * setup.sms < kKv8MaxCtas ? 2 * setup.sms : kKv8MaxCtas;
  if (ctas > items * item_tiles) ctas = items * item_tiles;
  kv8_config(cfg, attr, dim3(unsigned(ctas)), Cfg::kThreads, Cfg::kSmem, s, 0);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_kv8_attn<HD, HB, false>, k, a);
  if (e != cudaSuccess || ctas < 2) return e;
  // (the last CTA's items end with it)
  // a warp per row where there are many rows, up to a block's eight where there are few (1 x 131077 positions, 64/8 heads, eight:
  // 48.7 us, one: 56.7; 56 ragged, 32/8, by this rule: 92.2, eight: 92.9, one: 94.2)
  const int64_t cuts = ctas - 1 < items ? ctas - 1 : items, rows = a.G;
  int per = kKv8MergeWarps;
  while (per > 1 && cuts * ((rows * per + kKv8MergeWarps - 1) / kKv8MergeWarps) > 4 * setup.sms) per /= 2;
  kv8_config(cfg, attr, dim3(unsigned(cuts), unsigned((rows * per + kKv8MergeWarps - 1) / kKv8MergeWarps)), 32 * kKv8MergeWarps, 0, s, 0);
  return cudaLaunchKernelEx(&cfg, k_kv8_merge<HD>, k, a, int(ctas), int(Cfg::kPart), HB, per);
}

template <int HD>
static cudaError_t kv8_launch_attn(const Kv4& k, const Kv8AttnArgs& a, int64_t item_tiles, cudaStream_t s) {
  if (a.G <= 2) return kv8_launch_attn<HD, 2>(k, a, item_tiles, s);
  if (a.G <= 4) return kv8_launch_attn<HD, 4>(k, a, item_tiles, s);
  return a.G <= 8 ? kv8_launch_attn<HD, 8>(k, a, item_tiles, s) : kv8_launch_attn<HD, 16>(k, a, item_tiles, s);
}

}  // namespace nt

using namespace nt;

extern "C" nt_status nt_attention_kv8(const nt_kv8_cache* c, int32_t layer, int32_t n_heads, int32_t n, const int32_t* dev_seq,
                                      const int32_t* dev_ctx, int32_t n_select, const int32_t* dev_pages, const float* dev_q,
                                      int64_t q_stride, float* dev_out, int64_t out_stride, void* dev_workspace,
                                      size_t workspace_bytes, void* stream) {
  const char* who = "nt_attention_kv8";
  auto bad = [&](const char* what) { return fail(NT_E_INVAL, std::string(who) + ": " + what); };
  Kv4 k;
  nt_status st = kv8_check(c, who, true, &k);
  if (st) return st;
  if (layer < 0 || layer >= k.n_layers) return bad("layer out of range");
  if (n_heads < 1 || n_heads % k.n_kv) return bad("n_heads must be a positive multiple of n_kv_heads");
  const int G = n_heads / k.n_kv;
  if (G > kKv8MaxGroup) return fail(NT_E_UNSUPPORTED, std::string(who) + ": more than 16 query heads per kv head");
  if (n < 0 || n > 65536 || (!dev_seq && n > k.max_seqs)) return bad("n out of range");
  if (n_select < 0 || n_select > 65536) return bad("n_select outside [0, 65536]");
  const int64_t row = int64_t(n_heads) * k.hd;
  if (q_stride < row || out_stride < row || q_stride % 4 || out_stride % 4 || q_stride > (int64_t(1) << 40) ||
      out_stride > (int64_t(1) << 40))
    return bad("strides must be multiples of 4 and at least n_heads * head_dim");
  if (!kv4_aligned(dev_q, 16) || !kv4_aligned(dev_out, 16) || !kv4_aligned(dev_workspace, 16))
    return bad("q, out or workspace is NULL or not 16-byte aligned");
  if ((n_select && !kv4_aligned(dev_pages, 4)) || (dev_seq && !kv4_aligned(dev_seq, 4)) || (dev_ctx && !kv4_aligned(dev_ctx, 4)))
    return bad("a list is NULL or not 4-byte aligned");
  if (!n_select && dev_pages) return bad("pages without n_select");
  const size_t wb = kv8_attn_ws_bytes(k.hd);
  if (workspace_bytes < wb) return bad("workspace too small");
  if (n == 0) return NT_OK;
  const int64_t items = int64_t(n) * k.n_kv;
  const int64_t qb = ((n - 1) * q_stride + row) * 4, ob = ((n - 1) * out_stride + row) * 4, lb = int64_t(n) * 4;
  auto meets = [&](const void* p, int64_t bytes) {   // a written buffer and everything else
    return kv4_meets_cache(k, p, bytes) || kv4_overlap(p, bytes, dev_q, qb) || (dev_seq && kv4_overlap(p, bytes, dev_seq, lb)) ||
           (dev_ctx && kv4_overlap(p, bytes, dev_ctx, lb)) || (n_select && kv4_overlap(p, bytes, dev_pages, items * n_select * 4));
  };
  if (meets(dev_out, ob) || meets(dev_workspace, int64_t(wb)) || kv4_overlap(dev_out, ob, dev_workspace, int64_t(wb)))
    return bad("the output or the workspace overlaps another buffer");
  // a launch's tiles are counted in 32 bits
  const int64_t entry_pages = n_select && n_select < k.max_pages ? n_select : k.max_pages;
  const int64_t entry_tiles = int64_t(k.n_kv) * ((entry_pages * k.page_len + kKv8Tile - 1) / kKv8Tile), most = int64_t(1) << 30;
  if (entry_tiles > most) return bad("n_kv_heads * max_pages * page_len is too large");
  const int32_t batch = entry_tiles * kKv8Batch <= most ? kKv8Batch : int32_t(most / entry_tiles);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Kv8AttnArgs a{};
  a.layer = layer;
  a.G = G;
  a.k = n_select;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.scale = 1.4426950408889634f / sqrtf(float(k.hd));
  a.open = static_cast<int2*>(dev_workspace);
  a.part = static_cast<float*>(dev_workspace) + 2 * kKv8MaxCtas;
  for (int32_t i = 0; i < n; i += batch) {
    a.n = n - i < batch ? n - i : batch;
    a.seq0 = i;
    a.seq = dev_seq ? dev_seq + i : nullptr;
    a.ctx = dev_ctx ? dev_ctx + i : nullptr;
    a.pages = n_select ? dev_pages + int64_t(i) * k.n_kv * n_select : nullptr;
    a.q = dev_q + int64_t(i) * q_stride;
    a.out = dev_out + int64_t(i) * out_stride;
    const int64_t tiles = entry_tiles / k.n_kv;         // of an item, by capacity
    const cudaError_t e = k.hd == 64 ? kv8_launch_attn<64>(k, a, tiles, s) : kv8_launch_attn<128>(k, a, tiles, s);
    if (e != cudaSuccess) return cuda_fail(e, who);
  }
  return NT_OK;
}
