// nt_kv4_attn_tc.cu -- attention over the paged 4-bit K/V cache with the products on
// tcgen05: 8 or 16 query heads per kv head of 128 dimensions, work for the whole GPU.
//
// The mathematics and the share-out are nt_kv4_attn.cu's; what differs is who
// multiplies.  mma.sync takes the issue and FMA path of the warps that decode, so
// that with 8 heads decoding and products took turns.  Here four warps decode a tile of
// 128 positions straight into tensor memory, as the A operand of two products whose
// accumulators stand there too:
//   S^T [128 positions][16] = K [128][hd] . q^T,          16 columns: q hi, then q lo
//   O^T [128 dims][16]      = V^T [128][128 positions] . P^T,   P hi, then P lo
// (16 heads: hi and lo one after the other into the same 16 columns).  K and V^T are decoded from the same words by the
// same lanes as for mma.sync: a lane's pairs are its places in a 16 x 128-bit tile (tcgen05.st.16x128b).  q and P
// are the small operands, f16 in shared memory.  After S^T a thread holds the scores of its
// position for every head, after O^T the sums of its dimension for every head:
// the running sums are its own registers, added with ordinary rounding tile by tile.
//
// A group is four such warps and a fifth that copies tiles and starts products; groups run by themselves, so that one
// decodes while another waits for its products.  With 8 heads four groups fit an SM: the scores stand where V^T will,
// the outputs where K was, 128 of the 512 columns a group; with 16 heads the registers allow three, which need not share.
// The fifth warps give registers up to the others (setmaxnreg).
//
// What bounds it: issue slots and waits.  A tile costs each of the four warps 800 instructions (26.3 M in all for 8192 tiles),
// over half of them decoding, and the SM's 4 groups take 0.52 us a tile together, of which the instructions are 0.39; issue is
// 68% busy, the start included.  (Registers spill: 60 bytes stored and 40 loaded with 8 heads, 24 and 12 with 16.)  The
// start is 10 us: lengths, pages and first tiles one after the other, and a second launch merges partial results.
// 131077 positions of 8 kv heads (151 MB): 38.7 us, with mma.sync 43.6; 4 x 40000 of 4 kv heads with 16 heads each 37.4
// and 46.8; 4 x 20000 of 8 29.8 and 31.8; 16 of up to 4000 22.8 and 23.1; 64 of up to 1000 26.5 and 26.2.
// (On the way, for the first: three groups, a warp of theirs starting products by its thread 0: 62.0; by an elected
// thread: 54.8; a fifth warp for it: 44.5; that warp awaiting K by an mbarrier, q in one pass: 42.4; four groups: 40.6.)
#include "nt_kv4_attn.cuh"

namespace nt {

constexpr int kTcTile = 128;             // positions of a tile: 8 chunks
// An item's start and end, in tiles.  (At 1, 2 and 3: 131077 positions of 8 kv heads 40.6, 39.5, 39.4 us; 64 of up to 1000
// 27.9, 27.3, 27.5; 16 of up to 4000 22.7, 23.4, 22.8.)
constexpr int kTcItemTiles = 2;

template <int HB>
struct Kv4TcCfg {
  static constexpr int HD = 128, N = 16, kRowBlocks = HB / 4, CB = kv4_chunk_bytes(HD);
  static constexpr int kGroups = HB == 8 ? 4 : 3, kWarps = 4 * kGroups;   // warps that decode
  static constexpr int kThreads = 128 * (kGroups + 1);                    // and one of each that copies and starts products
  static constexpr int S = 2;                                       // ring stages of a group
  static constexpr int kRegs = HB == 8 ? 112 : 152, kHelpRegs = HB == 8 ? 32 : 56;   // the launch's, shared out again
  static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
  static_assert(kGroups * kRegs + kHelpRegs <= (kGroups + 1) * kLaunchRegs, "an increase past the launch's waits for ever");
  static_assert(kHelpRegs < kLaunchRegs && kLaunchRegs < kRegs, "the helpers give, the others take");
  static constexpr int kTileBytes = 8 * CB;
  static constexpr int kPart = kv4_part_floats(HD, HB);
  // B operands, 8 x 8 blocks of 128 bytes: [N / 8][k / 8].  A block of q holds 8 rows (N) of 8 k, one of P 8 rows (k) of 8
  // heads: a thread, which has a position's weights, stores them as 16 bytes
  static constexpr int kStep = 128, kRows = 16 * kStep;
  // shared memory of a group
  static constexpr int kRing = 0;
  static constexpr int kQ = kRing + S * kTileBytes;
  static constexpr int kP = kQ + kRowBlocks * kRows;
  static constexpr int kSlot = kP + kRowBlocks * kRows;
  static constexpr int kRed = kSlot + kPart * 4;                    // [4][HB] maxima of the warps
  static constexpr int kBars = kRed + 4 * HB * 4;                   // full [S], scores, outputs, keys
  static constexpr int kMiss = kBars + 8 * (S + 3);                 // [S]: the tile lacks a page
  static constexpr int kGroup = (kMiss + 4 * S + 127) / 128 * 128;
  // of the CTA
  static constexpr int kPrefix = kGroups * kGroup;
  static constexpr int kEntry = kPrefix + (kKv4Batch + 4) * 4;
  static constexpr int kItem = kEntry + kKv4Batch * 8;
  static constexpr int kOrder = kItem + 2 * kGroups * 4;
  static constexpr int kTmem = kOrder + kWarps * 32 * 4;
  static constexpr int kSmem = kTmem + 16;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  static_assert(kPart * 4 <= S * kTileBytes, "a group's ring holds a partial result");
  // tensor memory of a group, in columns.  HB 8: the scores stand where V^T will, the outputs where K was
  static constexpr int kColK = 0, kColV = 64, kColS = HB == 8 ? 64 : 128, kColO = HB == 8 ? 0 : 144;
  static constexpr int kCols = HB == 8 ? 128 : 160;
  static_assert(kGroups * kCols <= 512, "tensor memory of an SM");
};

// ------------------------------------------------------------ tcgen05 pieces --

// The B operand at a: blocks of 8 k 128 bytes apart, of 8 rows 16 such, no swizzle (the same for both orders within a block).
__device__ __forceinline__ uint64_t kv4_tc_desc(uint32_t a) {
  return uint64_t((a & 0x3ffffu) >> 4) | uint64_t(128 >> 4) << 16 | uint64_t(2048 >> 4) << 32 | uint64_t(1) << 46;
}
__device__ __forceinline__ void kv4_tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
      : "memory");
}
__device__ __forceinline__ void kv4_tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// 16 rows x 64 columns: lane (gi, tg) has columns 4 i + tg of rows gi (r[2 i]) and gi + 8 (r[2 i + 1])
__device__ __forceinline__ void kv4_tc_st16(uint32_t a, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// 16 rows x 32 columns
__device__ __forceinline__ void kv4_tc_st8(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// this lane's row, 16 columns
__device__ __forceinline__ void kv4_tc_ld16(uint32_t a, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
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
// Barrier of a group's 128 threads; whether any of them says so.
template <int THREADS>
__device__ __forceinline__ bool kv4_group_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.or.pred q, %1, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(uint32_t(p)), "n"(THREADS)
      : "memory");
  return r;
}

// ------------------------------------------------------------ the kernel --

template <int HB>
__global__ void __launch_bounds__(Kv4TcCfg<HB>::kThreads, 1) k_kv4_attn_tc(Kv4 c, Kv4AttnArgs a) {
  using Cfg = Kv4TcCfg<HB>;
  using L = Kv4Chunk<128>;
  constexpr int HD = 128, NG = 4, N = Cfg::N, S = Cfg::S, CB = Cfg::CB;
  extern __shared__ __align__(128) uint8_t sm[];
  int* prefix = reinterpret_cast<int*>(sm + Cfg::kPrefix);
  int2* entry = reinterpret_cast<int2*>(sm + Cfg::kEntry);
  int* slot_item = reinterpret_cast<int*>(sm + Cfg::kItem);
  const int t = threadIdx.x, warp = __shfl_sync(0xffffffffu, t >> 5, 0), lane = t & 31;
  const bool helps = warp >= Cfg::kWarps;
  const int group = helps ? (warp - Cfg::kWarps) % Cfg::kGroups : warp >> 2;   // the last warp has nothing to do
  constexpr int G = HB;
  const int n = a.n;
  uint8_t* gs = sm + group * Cfg::kGroup;
  auto slot_ptr = [&](int w) {
    return reinterpret_cast<float*>(sm + (w >> 1) * Cfg::kGroup + (w & 1 ? Cfg::kRing : Cfg::kSlot));
  };
  const uint32_t gsm = kv4_smem(gs), bars = gsm + Cfg::kBars, bar_s = bars + 8 * S, bar_o = bar_s + 8, bar_k = bar_o + 8;
  volatile uint32_t* miss = reinterpret_cast<volatile uint32_t*>(gs + Cfg::kMiss);

  if (helps && warp < Cfg::kWarps + Cfg::kGroups && lane < S + 3) kv4_bar_init(bars + 8 * lane, lane == S + 2 ? 4 : 1);
  if (t < 2 * Cfg::kGroups) slot_item[t] = -1;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncthreads();   // barriers
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // Tensor memory is taken only now, though 0.3 us earlier would be for nothing: a kernel that this one waits for could want
  // it on this SM.  The other fifth warps hear of it before they copy, those that decode with their first tile.
  if (warp == Cfg::kWarps)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(kv4_smem(sm + Cfg::kTmem))
                 : "memory");
  const volatile uint32_t* tensor_memory = reinterpret_cast<const volatile uint32_t*>(sm + Cfg::kTmem);
  kv4_count<Cfg::kThreads / 32>(c, a, kTcTile, kTcItemTiles, prefix, entry, reinterpret_cast<int*>(sm + Cfg::kOrder));
  const int total = prefix[n], groups = int(gridDim.x) * Cfg::kGroups;
  int share = (total + groups - 1) / groups;
  if (share < 1) share = 1;
  const int c0 = int(blockIdx.x) * Cfg::kGroups * share;
  const int c1 = c0 + Cfg::kGroups * share < total ? c0 + Cfg::kGroups * share : total;
  float* part0 = a.part + int64_t(blockIdx.x) * 2 * Cfg::kPart;
  int* header = reinterpret_cast<int*>(part0 + 2 * Cfg::kPart - 4);
  if (t == 0) header[0] = -1;
  asm volatile("griddepcontrol.launch_dependents;");
  kv4_empty_entries(c, a, entry, HD);

  const int w0 = c0 + group * share;
  const int count = w0 >= c1 ? 0 : (w0 + share > c1 ? c1 - w0 : share);
  const int cpp = c.page_len / kKv4Chunk;
  const uint8_t* layer_pool = c.pool + int64_t(a.layer) * c.n_pages * c.page_bytes();
  auto tiles = [&](int len) { return (len + kTcTile - 1) / kTcTile; };
  // the item of unit y: entry e, kv head g, tile ti of nt (below 0: the item's cost, nothing to read)
  auto locate = [&](int y, int& e, int& g, int& ti, int& nt) {
    e = kv4_find(prefix, n, y);
    nt = tiles(entry[e].y);
    const int r = y - prefix[e], units = nt + kTcItemTiles;
    g = int(unsigned(r) / unsigned(units));
    ti = r - g * units - kTcItemTiles;
  };
  // chunk ch of unit x of this group, as an index within the layer's pool; -1: no page, -2: behind the end, -3: no tile
  auto resolve = [&](int x, int ch) -> int {
    if (x >= count) return -3;
    int e, g, ti, nt;
    locate(w0 + x, e, g, ti, nt);
    if (ti < 0) return -3;
    const int ci = 8 * ti + ch;
    if (ci * kKv4Chunk >= entry[e].y) return -2;
    const int page = c.table[int64_t(entry[e].x) * c.max_pages + unsigned(ci) / unsigned(cpp)];
    if (page < 0 || page >= c.n_pages) { kv4_flag(c, NT_KV4_BAD_PAGE); return -1; }
    return (page * c.n_kv + g) * cpp + int(unsigned(ci) % unsigned(cpp));
  };

  constexpr uint32_t kIdesc = 1u << 4 | uint32_t(N / 8) << 17 | uint32_t(128 / 16) << 24;   // fp32 += f16 f16, 128 x N
  const int alone = 1 + group, all = 1 + Cfg::kGroups + group;   // barriers: of the warps that decode, of the whole group
  int k = 0, e = 0, g = 0, ti0 = 0, nt = 1;
  bool dead = false;   // a wait ran out: nothing more is copied or multiplied (the same in all of the group)
  if (count > 0) locate(w0, e, g, ti0, nt);

  if (helps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kHelpRegs));
    kv4_tc_before();
    asm volatile("barrier.cta.sync.aligned 14, 128;" ::: "memory");
    kv4_tc_after();
    const uint32_t tmem = *tensor_memory + group * Cfg::kCols;
    if (warp < Cfg::kWarps + Cfg::kGroups) {
      // Copies: the group's tile x (an item's cost is none) into stage x % S, whose barrier phase x / S completes.  A lane
      // knows chunk lane % 8 of unit 4 b + lane / 8: addr those of the units up to the next multiple of 4, next four more.
      int unit = 0, issued = 0, addr = resolve(lane >> 3, lane & 7), next = -3, known = 4;
      auto ahead = [&]() {
        if (unit <= known - 4) return;
        next = resolve(known + (lane >> 3), lane & 7);
        known += 4;
      };
      auto issue = [&]() {
        while (unit < count && !dead) {
          if ((unit & 3) == 0 && unit) {
            ahead();
            addr = next;
          }
          const int x = __shfl_sync(0xffffffffu, addr, 8 * (unit & 3) + (lane & 7)), st = issued % S;
          unit++;
          if (__any_sync(0xffffffffu, x == -3)) continue;
          const uint32_t have = __ballot_sync(0xffffffffu, lane < 8 && x >= 0);
          const bool lacks = __any_sync(0xffffffffu, x == -1);
          const uint32_t bar = bars + 8 * st;
          if (lane == 0) {
            miss[st] = lacks;
            if (lacks) kv4_bar_arrive(bar);
            else kv4_bar_expect(bar, uint32_t(__popc(have)) * CB);
          }
          __syncwarp();
          if (!lacks && lane < 8 && x >= 0)
            kv4_copy(gsm + Cfg::kRing + st * Cfg::kTileBytes + lane * CB, layer_pool + int64_t(x) * CB, CB, bar);
          issued++;
          return;
        }
      };
#pragma unroll 1
      for (int i = 0; i < S; i++) issue();
      int x = 0;   // tiles behind
#pragma unroll 1
      while (k < count) {
        for (; ti0 < 0 && k < count; ti0++) k++;
        if (k == count) break;
        const int seg = nt - ti0 < count - k ? nt - ti0 : count - k;
#pragma unroll 1
        for (const int k1 = k + seg; k < k1; k++, x++) {
          if (dead) continue;
          const bool lacks = miss[x % S], came = __all_sync(0xffffffffu, kv4_bar_wait(bar_k, uint32_t(x) & 1u));
          if (came && !lacks) {
            kv4_tc_after();
            if (kv4_elect()) {
#pragma unroll
              for (int y = HB / 8 - 1; y >= 0; y--)   // HB 16: lo, then hi
#pragma unroll
                for (int kk = 0; kk < 8; kk++)
                  kv4_tc_mma(tmem + Cfg::kColS, tmem + Cfg::kColK + 8 * kk,
                             kv4_tc_desc(gsm + Cfg::kQ + y * 2 * Cfg::kRows + kk * 2 * Cfg::kStep), kIdesc,
                             kk > 0 || y < HB / 8 - 1);
              kv4_tc_commit(bar_s);
            }
            __syncwarp();
          }
          ahead();
          if (kv4_group_any<160>(all, !came)) {
            dead = kv4_group_any<160>(all, !came);
            if (!dead) kv4_group_any<160>(all, false);
          }
          if (!dead && !lacks) {
            kv4_tc_after();
            if (kv4_elect()) {
#pragma unroll
              for (int y = HB / 8 - 1; y >= 0; y--)   // HB 16: lo, then hi
#pragma unroll
                for (int kk = 0; kk < 8; kk++)
                  kv4_tc_mma(tmem + Cfg::kColO, tmem + Cfg::kColV + 8 * kk,
                             kv4_tc_desc(gsm + Cfg::kP + y * 2 * Cfg::kRows + kk * 2 * Cfg::kStep), kIdesc | 1u << 16,
                             kk > 0 || y < HB / 8 - 1);
              kv4_tc_commit(bar_o);
            }
            __syncwarp();
          }
          issue();   // every warp has read the tile: its stage takes the next one
        }
        if (k < count) locate(w0 + k, e, g, ti0, nt);
      }
      if (dead)   // copies in flight land before the shared memory is given up
        for (int y = issued < S ? 0 : issued - S; y < issued; y++) kv4_bar_wait(bars + 8 * (y % S), uint32_t(y / S) & 1u);
    }
    kv4_tc_before();
    asm volatile("barrier.cta.sync.aligned 15, %0;" ::"n"(Cfg::kThreads) : "memory");
    if (warp == Cfg::kWarps) {
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(*tensor_memory));
    }
    return;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kRegs));

  const int tid = t & 127, wq = warp & 3, gi = lane >> 2, tg = lane & 3;
  const uint32_t mine = uint32_t(32 * wq) << 16;   // this warp's rows
  float O[HB], l[HB], mref[HB], cs[HB];
  uint32_t ps = 0, po = 0;      // parities of the products' barriers
  int tile_no = 0;              // tiles behind
  uint32_t tmem = 0;            // known with the first tile
  bool pending = false;         // an O^T has been started and not been taken in

  // adds the last tile's outputs to the sums; false: they never came
  auto take = [&]() -> bool {
    if (!pending) return true;
    pending = false;
    const bool ok = kv4_bar_wait(bar_o, po);
    po ^= 1u;
    kv4_tc_after();
    float v[N];
    kv4_tc_ld16(tmem + mine + Cfg::kColO, v);
#pragma unroll
    for (int h = 0; h < HB; h++) O[h] += HB == 8 ? v[h] + v[(8 + h) % N] : v[h];
    return ok;
  };

#pragma unroll 1
  while (k < count) {
    for (; ti0 < 0 && k < count; ti0++) k++;
    if (k == count) break;
    const int seg = nt - ti0 < count - k ? nt - ti0 : count - k;
    int live = entry[e].y - ti0 * kTcTile;
    bool poison = false;
    {
      // q, a head by one warp: scaled (as in nt_kv4_attn.cu) so that its largest element is in [2^10, 2^12), split
      const float* qb = a.q + int64_t(e) * a.q_stride + int64_t(g) * G * HD;
      float* red = reinterpret_cast<float*>(gs + Cfg::kRed);
#pragma unroll
      for (int i = 0; i < HB / 4; i++) {
        const int h = 4 * i + wq;
        const float4 u = *reinterpret_cast<const float4*>(qb + h * HD + 4 * lane);
        float top = fmaxf(fmaxf(fabsf(u.x), fabsf(u.y)), fmaxf(fabsf(u.z), fabsf(u.w)));
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        int ex = int(__float_as_uint(top) >> 23);
        ex = ex < 14 ? 14 : ex;                                       // (zeros and values below 2^-113)
        const float up = __uint_as_float(uint32_t(264 - ex) << 23) * a.q_scale;   // 2^(137 - ex) q_scale
        if (lane == 0) red[h] = __uint_as_float(uint32_t(ex - 13) << 23);         // 2^(ex - 140)
        // dimension 32 j + 8 tg + 4 b + p is row 32 j + 8 p + 2 tg + b of the product: K's pairs
        const float x[4] = {u.x * up, u.y * up, u.z * up, u.w * up};
        const int row = 2 * ((lane >> 1) & 3) + (lane & 1);
        uint8_t* at = gs + Cfg::kQ + (lane >> 3) * 4 * Cfg::kStep + (h & 7) * 16 + row * 2;
#pragma unroll
        for (int p = 0; p < 4; p++) {
          const __half hi = __float2half_rn(x[p]), lo = __float2half_rn(x[p] - __half2float(hi));
          *reinterpret_cast<__half*>(at + p * Cfg::kStep + (h >> 3) * Cfg::kRows) = hi;
          *reinterpret_cast<__half*>(at + p * Cfg::kStep + ((HB + h) >> 3) * Cfg::kRows) = lo;
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      kv4_group_any<128>(alone, false);
#pragma unroll
      for (int h = 0; h < HB; h++) {
        cs[h] = red[h];
        O[h] = l[h] = 0.f;
        mref[h] = -3e38f;
      }
    }

#pragma unroll 1
    for (const int k1 = k + seg; k < k1; k++, tile_no++, live -= kTcTile) {
      const int st = tile_no % S;
      if (dead) continue;
      bool fail = !__all_sync(0xffffffffu, kv4_bar_wait(bars + 8 * st, uint32_t(tile_no / S) & 1u));
      uint8_t* tile = gs + Cfg::kRing + st * Cfg::kTileBytes;
      const uint32_t base = kv4_smem(tile);
      const bool lacks = fail || miss[st];
      if (tile_no == 0) {
        kv4_tc_after();
        tmem = *tensor_memory + group * Cfg::kCols;
      }
      // ---- K of chunks 2 wq and 2 wq + 1: rows are positions
      if (!lacks) {
#pragma unroll
        for (int u = 0; u < 2; u++) {
          const uint32_t ch = base + (2 * wq + u) * CB;
          uint32_t r[32];
#pragma unroll
          for (int i = 0; i < 2; i++) {
            uint32_t w[NG];
            kv4_words<NG>(ch + (i * 32 + lane) * (4 * NG), w);
            const uint2 s2 = kv4_lds8(ch + L::kKS + (8 * i + gi) * (2 * NG));
            const uint32_t ks[2] = {s2.x, s2.y}, ks72[2] = {kv4_h2mul(s2.x, kMinus72), kv4_h2mul(s2.y, kMinus72)};
#pragma unroll
            for (int j = 0; j < NG; j++) {
              uint32_t b[4];
              kv4_decode(w[j], kv4_half(ks[j >> 1], j & 1), kv4_half(ks72[j >> 1], j & 1), b);
#pragma unroll
              for (int p = 0; p < 4; p++) r[2 * (4 * j + p) + i] = b[p];
            }
          }
          if (HB == 8 && u == 0) fail = !take() || fail;    // outputs share K's columns
          kv4_tc_st16(tmem + mine + (uint32_t(16 * u) << 16) + Cfg::kColK, r);
        }
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      kv4_tc_before();
      __syncwarp();
      if (lane == 0) kv4_bar_arrive(bar_k);
      if (lacks) {
        if (HB == 8) fail = !take() || fail;
        if (kv4_group_any<160>(all, fail)) {
          dead = kv4_group_any<160>(all, fail);
          if (!dead) kv4_group_any<160>(all, false);
        }
        poison = true;
        continue;
      }
      if (HB == 16) fail = !take() || fail;   // before V^T moves in
      if (live < kTcTile) {   // positions behind the end: scale 0 (of this warp's dimensions), whatever the page holds there
        for (int p = live + lane; p < kTcTile; p += 32)
          *reinterpret_cast<uint16_t*>(tile + (p >> 4) * CB + L::v_scale(p & 15, wq)) = 0;
        __syncwarp();
      }
      // ---- scores of position tid
      float x[HB];
      auto scores = [&]() {
        fail = !kv4_bar_wait(bar_s, ps) || fail;
        ps ^= 1u;
        kv4_tc_after();
        float v[N];
        kv4_tc_ld16(tmem + mine + Cfg::kColS, v);
#pragma unroll
        for (int h = 0; h < HB; h++) x[h] = HB == 8 ? v[h] + v[(8 + h) % N] : v[h];
      };
      // ---- V^T: rows are dimensions 32 wq + 4 gi + y (row 8 y + gi of the warp's), columns pairs of positions
#pragma unroll
      for (int half = 0; half < 2; half++) {
        uint32_t ra[16], rb[16];
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const int cc = 4 * half + (i >> 1), r = i & 1;
          const uint32_t ch = base + cc * CB;
          const uint32_t w = kv4_lds4(ch + L::kV + (r * 32 + lane) * (4 * NG) + 4 * wq);
          const uint32_t d = kv4_lds4(ch + L::kVS + (r * 4 + tg) * (4 * NG) + 4 * wq);
          uint32_t b[4];
          kv4_decode(w, d, kv4_h2mul(d, kMinus72), b);
          ra[2 * i] = b[0]; ra[2 * i + 1] = b[1];
          rb[2 * i] = b[2]; rb[2 * i + 1] = b[3];
        }
        if (HB == 8 && half == 0) scores();   // V^T goes where they stood
        kv4_tc_st8(tmem + mine + Cfg::kColV + 32 * half, ra);
        kv4_tc_st8(tmem + mine + (16u << 16) + Cfg::kColV + 32 * half, rb);
      }
      if (HB != 8) scores();
      if (live < kTcTile) {
#pragma unroll
        for (int h = 0; h < HB; h++) x[h] = tid < live ? x[h] : -INFINITY;
      }
      // ---- weights, as hi and lo rows of the B operand
      float p[HB], sum;
      auto weights = [&]() {
        sum = 0.f;
        uint8_t* at = gs + Cfg::kP + tid * 16;   // block tid / 8, its row tid % 8
#pragma unroll
        for (int b = 0; b < HB / 8; b++) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int h = 8 * b + 2 * i;
            p[h] = kv4_ex2(fmaf(x[h], cs[h], -mref[h]));
            p[h + 1] = kv4_ex2(fmaf(x[h + 1], cs[h + 1], -mref[h + 1]));
            sum += p[h] + p[h + 1];
            kv4_split(p[h], p[h + 1], hi[i], lo[i]);
          }
          *reinterpret_cast<uint4*>(at + b * Cfg::kRows) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(at + (HB / 8 + b) * Cfg::kRows) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      };
      weights();
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      kv4_tc_before();
      if (kv4_group_any<160>(all, !(sum <= 32768.f) || fail)) {
        // A weight may have passed 2^15 / HB (at first all are infinite; a NaN may hide one): the maxima over the tile's
        // positions.  One that passes its head's reference by 11 moves it, so that the next tile does not come here again.
        float* red = reinterpret_cast<float*>(gs + Cfg::kRed);
#pragma unroll
        for (int h = 0; h < HB; h++) {
          float top = x[h];
#pragma unroll
          for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          if (lane == 0) red[wq * HB + h] = top;
        }
        dead = kv4_group_any<160>(all, fail);
#pragma unroll
        for (int h = 0; h < HB; h++) {
          const float top = fmaxf(fmaxf(red[h], red[HB + h]), fmaxf(red[2 * HB + h], red[3 * HB + h])) * cs[h];
          const float to = top - mref[h] > 11.f ? top - 6.f : mref[h], f = kv4_ex2(mref[h] - to);
          mref[h] = to;
          l[h] *= f;
          O[h] *= f;
        }
        if (dead) continue;
        weights();
        kv4_tc_before();
        kv4_group_any<160>(all, false);
      }
      pending = true;
#pragma unroll
      for (int h = 0; h < HB; h++) l[h] += p[h];
    }
    // ---- the end of the segment: thread tid has dimension 32 wq + 4 (lane % 8) + lane / 8, its l that of position tid
    if (!take() || dead) poison = true;
    if (dead && tid == 0) kv4_flag(c, NT_KV4_TIMEOUT);
    float* red = reinterpret_cast<float*>(gs + Cfg::kRed);
#pragma unroll
    for (int h = 0; h < HB; h++) {
#pragma unroll
      for (int o = 16; o; o >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
      if (lane == 0) red[wq * HB + h] = l[h];
    }
    poison = kv4_group_any<128>(alone, poison);
    const bool whole = ti0 == 0 && seg == nt;
    const int slot = 2 * group + (ti0 > 0 ? 0 : 1), e_was = e, g_was = g;
    float* to = whole ? a.out + int64_t(e_was) * a.out_stride + int64_t(g_was) * G * HD : slot_ptr(slot);
    if (!whole && tid == 0) slot_item[slot] = e_was * c.n_kv + g_was;
    const int dim = 32 * wq + 4 * (lane & 7) + (lane >> 3);
#pragma unroll
    for (int h = 0; h < HB; h++) {
      float sum = (red[h] + red[HB + h]) + (red[2 * HB + h] + red[3 * HB + h]);
      if (poison) sum = NAN;
      to[h * HD + dim] = whole ? O[h] / sum : O[h];
      if (!whole && tid == 0) reinterpret_cast<float2*>(to + HB * HD)[h] = make_float2(mref[h], sum);
    }
    if (k < count) locate(w0 + k, e, g, ti0, nt);
    kv4_group_any<128>(alone, false);   // red is read
  }
  kv4_tc_before();
  asm volatile("barrier.cta.sync.aligned 15, %0;" ::"n"(Cfg::kThreads) : "memory");
  kv4_merge<HD, HB, Cfg::kWarps, 2 * Cfg::kGroups>(
      c, a, slot_item, slot_ptr, reinterpret_cast<int*>(sm + Cfg::kOrder) + (t >> 5) * 32,
      [&](int item, int& first, int& units) {
        const int ie = item / c.n_kv;
        units = tiles(entry[ie].y);
        first = prefix[ie] + item % c.n_kv * (units + kTcItemTiles) + kTcItemTiles;
      },
      c0, c1, Cfg::kGroups * share, part0, header);
}

template <int HB>
static cudaError_t kv4_launch_tc(const Kv4& k, const Kv4AttnArgs& a, int64_t most_units, cudaStream_t s, int* ctas) {
  using Cfg = Kv4TcCfg<HB>;
  static const KernelSetup setup = kernel_setup(k_kv4_attn_tc<HB>, Cfg::kSmem);
  if (setup.err != cudaSuccess) return setup.err;
  const int64_t useful = (most_units + Cfg::kGroups - 1) / Cfg::kGroups;
  int64_t n = setup.sms < kKv4AttnMaxCtas ? setup.sms : kKv4AttnMaxCtas;
  if (n > useful) n = useful;
  *ctas = int(n);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(n));
  cfg.blockDim = dim3(Cfg::kThreads);
  cfg.dynamicSmemBytes = Cfg::kSmem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_kv4_attn_tc<HB>, k, a);
}

// The registers that a block shares out again have to be those it is launched with: an increase past them waits for ever.
template <int HB>
static bool kv4_tc_runs() {
  cudaFuncAttributes f;
  if (cudaFuncGetAttributes(&f, k_kv4_attn_tc<HB>) == cudaSuccess) return f.numRegs == Kv4TcCfg<HB>::kLaunchRegs;
  cudaGetLastError();
  return false;
}
bool kv4_attn_tc_runs(int G) {
  static const bool runs[2] = {kv4_tc_runs<8>(), kv4_tc_runs<16>()};
  return runs[G == 16];
}

cudaError_t kv4_launch_attn_tc(const Kv4& k, const Kv4AttnArgs& a, cudaStream_t s, int* ctas) {
  const int64_t units = int64_t(a.n) * k.n_kv * ((int64_t(k.max_pages) * k.page_len + kTcTile - 1) / kTcTile + kTcItemTiles);
  return a.G == 8 ? kv4_launch_tc<8>(k, a, units, s, ctas) : kv4_launch_tc<16>(k, a, units, s, ctas);
}

}  // namespace nt
