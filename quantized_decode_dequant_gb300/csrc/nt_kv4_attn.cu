// nt_kv4_attn.cu -- GQA decode attention over the paged 4-bit K/V cache.
//
// out_j = sum_t softmax(q_j . K_t / sqrt(hd))_t V_t for the G query heads j of a
// kv head, in one pass over its chunks of 16 positions with a running maximum
// and sum (flash decoding): each warp copies its chunks from the pages into a
// ring of its own in shared memory (one bulk copy of 18 hd contiguous bytes per
// chunk), decodes codes in registers and contracts them on the tensor cores.
//
// Decoding.  Four bits moved to bits 4..7 of an f16 whose upper bits are 0x5400
// are the number 64 + q; one fused multiply-add gives the value, (64 + q) d - 72 d
// = d (q - 8), exactly: d has seven significant bits, so 72 d has eleven.  That is
// 3 shifts, 4 logic ops and 4 half2 multiply-adds for 8 values, the scale included.
// The words are laid out so that what a lane decodes is its own fragment of the
// B operand of mma.sync m16n8k16: nothing passes through shared memory twice.
//
// Contractions (G > 4; below 5 heads see N4).  Scores S[h][t] = q_h . K_t and outputs O[h][d] = sum_t P[h][t]
// V_t[d].  q (scaled) and P are split into two f16 terms, hi =
// f16(x) and lo = f16(x - hi), about 22 bits.  With G <= 8 hi takes rows 0..7 of
// the 16-row A operand of the scores and lo rows 8..15 (G = 16: a product each); for
// the outputs V^T is the A operand, 16 dimensions a tile, and P, as the scores'
// accumulators hold it, the B operand of 8 heads, hi and lo a product each into
// the same accumulators: 32 registers of them for 8 heads of 128 dimensions.
//
// With G <= 4 the positions are the rows of the scores' A operand and the heads the
// columns of B, hi of 4 heads and lo of 4 heads side by side, and the weights are
// transposed in registers (movmatrix) to be B of the outputs: half the products.
//
// What bounds it.  A byte of cache is 1.8 values; 8 values cost a lane 7 shifts and logic ops, 5 half2 ops and a sixteenth
// of a matrix product or more, and on this GPU mma.sync m16n8k16 (8 cycles of a sub-core) and the half2 ops (2) do
// not overlap.  With 4 heads that is just behind the memory: 56 sequences of up to 9001 positions of 8 kv heads
// (293 MB) take 65.1 us, 4.5 TB/s in all and 5.9 while data flows.  With 8 heads the products are twice as many
// and decide (43.6 us for 131077 positions where memory wants 22.3), so long work of 8 and 16 heads of
// 128 dimensions goes to the tcgen05 kernel of nt_kv4_attn_tc.cu (38.7 us).  Short work keeps to this kernel's cluster
// form: its warps go about alone, and there a first result counts, not a rate.
#include <cooperative_groups.h>

#include "nt_kv4_attn.cuh"

namespace nt {

constexpr int kKv4MinPairs = 1;        // fewest pairs of chunks of a warp: below, fewer CTAs work
// An item's start and end cost a warp about as much as a pair (q to split, sums to
// reduce, results to store): the share-out counts it as so many pairs more, in
// front of the item's own.  (Measured, with 1, 2 and 3: 56 sequences of up to 9001
// positions 66.4, 65.4, 65.0 us; 50 of 3000 with heads of 64 32.3, 32.1, 32.1; 64 of 200 12.6, 12.4, 14.6; 64 of
// up to 200 10.9, 14.0, 12.9; 64 of 700 22.7, 22.6, 24.2.)
constexpr int kKv4ItemPairs = 2;

// HB: query heads of a kv head that the instantiation is made for, up to 4, 8 or 16.
template <int HD, int HB>
struct Kv4AttnCfg {
  static constexpr int NW = HB == 16 ? (HD == 128 ? 8 : 12) : (HD == 128 && HB == 8 ? 12 : 16);   // warps: registers decide
  static constexpr int S = HD == 128 ? 2 : 4;                                          // ring stages of a warp
  static constexpr int kThreads = 32 * NW;
  static constexpr int kRows = HB;                                                     // heads of a partial result
  static constexpr int kPart = kv4_part_floats(HD, kRows);
  static constexpr int kPair = 2 * kv4_chunk_bytes(HD);                                // a stage: two chunks
  static constexpr int kRing = 0;
  static constexpr int kSlots = kRing + NW * S * kPair;                                // a slot of each warp (see below)
  static constexpr int kAcc = kSlots + NW * kPart * 4;                                 // sums of outputs, a warp's lane by lane
  static constexpr int kPrefix = kAcc + NW * kRows * HD * 4;
  static constexpr int kEntry = kPrefix + (kKv4Batch + 4) * 4;                         // {sequence, length} of each
  static constexpr int kBars = kEntry + kKv4Batch * 8;
  static constexpr int kItem = kBars + NW * S * 8;                                     // item of each slot (-1: none)
  static constexpr int kLane = kItem + 2 * NW * 4;                                     // [NW][2][32] words of the lanes
  static constexpr int kSmem = kLane + NW * 64 * 4;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  static_assert(kPart * 4 <= S * kPair && kPart % 4 == 0, "a warp's ring holds a partial result");
  static_assert(2 * NW <= 32, "a lane per slot");
  static_assert((S & (S - 1)) == 0, "stages are found by masks");
};

size_t kv4_attn_ws_bytes(int n_heads, int n_kv, int hd) {
  return size_t(kKv4AttnMaxCtas) * 2 * size_t(kv4_part_floats(hd, n_heads / n_kv > 8 ? 16 : (n_heads / n_kv > 4 ? 8 : 4))) * 4;
}

__device__ __forceinline__ void kv4_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 x 8 transpose of f16 held as matrix fragments (a row of two per lane)
__device__ __forceinline__ uint32_t kv4_transpose(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ int kv4_pairs(int len) { return (len + 2 * kKv4Chunk - 1) / (2 * kKv4Chunk); }

// ------------------------------------------------------------ the kernel --

// The chunk pairs of all (entry, kv head) items in a row, item after item, are
// shared out evenly: warp w of CTA b takes units [(b NW + w) C, (b NW + w + 1) C),
// a unit being a pair or an item's cost.
// An item that lies within a warp's share is finished by it; one that lies within
// a CTA's is merged in shared memory; the rest leaves partial results (at most two
// a CTA: slot 0 of an item begun before it, slot 1 of one that goes on behind it)
// to k_kv4_attn_merge.  Partial results are merged in the order of the positions,
// so the result does not depend on timing.  (WHOLE: CTA b's share is the items that begin in it; nothing is cut.)
//
// A warp leaves at most two partial results to the CTA: of the item it did not
// begin (slot 2 warp, in memory of its own) and of the one it did not end (slot
// 2 warp + 1, its last: it stands in the warp's ring, which is empty by then).
//
// CL: the form for few items whose capacity is small (see kv4_launch_attn).  A
// thread-block cluster has an item to itself, its warps share the pairs out, and
// the CTAs' partial results meet through distributed shared memory: no second launch,
// and no counting of the other entries.
template <int HD, int HB, bool CL, bool WHOLE = false>
__global__ void __launch_bounds__(Kv4AttnCfg<HD, HB>::kThreads, 1) k_kv4_attn(Kv4 c, Kv4AttnArgs a) {
  using Cfg = Kv4AttnCfg<HD, HB>;
  using L = Kv4Chunk<HD>;
  constexpr int NW = Cfg::NW, S = Cfg::S, NG = HD / 32, NT = HD / 8, CB = L::kBytes, ROWS = Cfg::kRows;
  constexpr bool N4 = HB == 4;             // hi and lo of up to 4 heads side by side as the 8 columns of a B operand
  constexpr int MT = HB == 16 ? 2 : 1;     // accumulators of 8 head columns each
  constexpr int NH = HB == 8 ? 1 : 2;      // heads whose scores a lane holds
  constexpr int NX = N4 ? 4 : 8;           // scores of a head and pair that a lane holds
  extern __shared__ __align__(128) uint8_t sm[];
  int* prefix = reinterpret_cast<int*>(sm + Cfg::kPrefix);
  int2* entry = reinterpret_cast<int2*>(sm + Cfg::kEntry);
  int* slot_item = reinterpret_cast<int*>(sm + Cfg::kItem);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, gi = lane >> 2, tg = lane & 3;
  const int G = a.G, n = a.n;
  auto slot_ptr = [&](int w) {
    return reinterpret_cast<float*>(w & 1 ? sm + Cfg::kRing + (w >> 1) * (S * Cfg::kPair) : sm + Cfg::kSlots + (w >> 1) * (Cfg::kPart * 4));
  };

  if (lane < S) kv4_bar_init(kv4_smem(sm + Cfg::kBars + (warp * S + lane) * 8));
  if (lane < 2) slot_item[2 * warp + lane] = -1;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- unit offsets of the entries (CL: the item's entry alone)
  if constexpr (CL) {
    uint32_t bad;
    const int2 sl = kv4_entry(c, a, int(blockIdx.y) / c.n_kv, &bad);
    if (bad && t == 0) kv4_flag(c, bad);
    if (t == 0) { entry[0] = sl; prefix[0] = 0; prefix[1] = kv4_pairs(sl.y); }
    __syncthreads();
  } else {
    kv4_count<NW>(c, a, 2 * kKv4Chunk, kKv4ItemPairs, prefix, entry, reinterpret_cast<int*>(sm + Cfg::kSlots));
  }
  const int e_own = CL ? int(blockIdx.y) / c.n_kv : 0, g_own = CL ? int(blockIdx.y) % c.n_kv : 0;
  auto ent = [&](int e) { return entry[CL ? 0 : e]; };   // sequence and length of entry e
  const int total = prefix[CL ? 1 : n], warps = int(gridDim.x) * NW;
  int share = (total + warps - 1) / warps;
  if (share < kKv4MinPairs) share = kKv4MinPairs;
  int c0 = int(blockIdx.x) * NW * share;                 // the CTA's first unit (total + 152 NW units fit an int)
  int c1 = c0 + NW * share < total ? c0 + NW * share : total;
  if constexpr (WHOLE) {   // the items that begin there, and a share of them for each warp; lane 1 looks for the end
    int y = lane == 1 ? c1 : c0;
    if (y < total) {
      const int e = kv4_find(prefix, n, y), units = kv4_pairs(entry[e].y) + kKv4ItemPairs;
      y = prefix[e] + int(unsigned(y - prefix[e] + units - 1) / unsigned(units)) * units;
    } else {
      y = total;
    }
    c0 = __shfl_sync(0xffffffffu, y, 0);
    c1 = __shfl_sync(0xffffffffu, y, 1);
    share = (c1 - c0 + NW - 1) / NW;
    if (share < kKv4MinPairs) share = kKv4MinPairs;
  }
  float* part0 = CL ? reinterpret_cast<float*>(sm + Cfg::kAcc) : a.part + int64_t(blockIdx.x) * 2 * Cfg::kPart;
  int* header = reinterpret_cast<int*>(part0 + 2 * Cfg::kPart - 4);   // of slot 1
  if (!CL && t == 0) header[0] = -1;
  asm volatile("griddepcontrol.launch_dependents;");
  if constexpr (CL) {
    if (total == 0) {   // no position: zeros, or NaN where the entry cannot be read
      if (blockIdx.x == 0)
        for (int x = t; x < G * HD; x += Cfg::kThreads)
          a.out[int64_t(e_own) * a.out_stride + int64_t(g_own) * G * HD + x] = ent(0).x < 0 ? NAN : 0.f;
      return;           // the whole cluster
    }
  } else {
    kv4_empty_entries(c, a, entry, HD);
    if (c0 >= c1) return;   // the whole CTA
  }

  const int w0 = c0 + warp * share;
  const int count = w0 >= c1 ? 0 : (w0 + share > c1 ? c1 - w0 : share);
  const uint32_t ring = kv4_smem(sm + Cfg::kRing) + uint32_t(warp) * (S * Cfg::kPair);
  const uint32_t bars = kv4_smem(sm + Cfg::kBars) + uint32_t(warp) * S * 8;
  const int cpp = c.page_len / kKv4Chunk;
  const uint8_t* layer_pool = c.pool + int64_t(a.layer) * c.n_pages * c.page_bytes();

  // the item of unit y of the share-out: entry e, kv head g, pair pi of np (below 0: the item's cost, nothing to read)
  auto locate = [&](int y, int& e, int& g, int& pi, int& np) {
    if constexpr (CL) {
      e = e_own; g = g_own; pi = y; np = total;
      return;
    }
    e = kv4_find(prefix, n, y);
    np = kv4_pairs(entry[e].y);
    const int r = y - prefix[e], units = np + kKv4ItemPairs;
    g = int(unsigned(r) / unsigned(units));
    pi = r - g * units - kKv4ItemPairs;
  };
  // indexes of the two chunks of pair x of this warp within the layer's pool (in
  // chunks); -1: no page, -2: behind the sequence's end, -3: no pair
  auto resolve = [&](int x) -> int2 {
    if (x >= count) return make_int2(-2, -2);
    int e, g, pi, np;
    locate(w0 + x, e, g, pi, np);
    if (pi < 0) return make_int2(-3, -3);
    const int len = ent(e).y;
    const int32_t* row = c.table + int64_t(ent(e).x) * c.max_pages;
    auto chunk = [&](int ci) -> int {
      if (ci * kKv4Chunk >= len) return -2;   // (len is at most 2^31 - 256)
      const int page = row[unsigned(ci) / unsigned(cpp)];
      if (page < 0 || page >= c.n_pages) { kv4_flag(c, NT_KV4_BAD_PAGE); return -1; }
      return (page * c.n_kv + g) * cpp + int(unsigned(ci) % unsigned(cpp));
    };
    return make_int2(chunk(2 * pi), chunk(2 * pi + 1));
  };

  int e = 0, g = 0, pi0 = 0, np = 1;
  if (count > 0) locate(w0, e, g, pi0, np);
  // Pair x stands in stage x % S and completes that stage's barrier phase x / S.
  int2 addr = resolve(lane);                  // of pairs 32 b + lane
  int issued = 0;
  uint32_t missing = 0;                       // bit per stage: it lacks a page
  constexpr uint32_t kDead = 1u << 31;        // a wait ran out: nothing more is copied or read
  constexpr uint32_t kHeld = 1u << 30;        // sums of the item's outputs are held in shared memory
  auto issue = [&]() {
    if (issued >= count || (missing & kDead)) return;
    if ((issued & 31) == 0 && issued) addr = resolve(issued + lane);
    const int x0 = __shfl_sync(0xffffffffu, addr.x, issued & 31), x1 = __shfl_sync(0xffffffffu, addr.y, issued & 31);
    const int at = issued & (S - 1);
    const bool lacks = x0 < 0 || x1 == -1;
    missing = lacks ? missing | (1u << at) : missing & ~(1u << at);
    if (lane == 0) {
      const uint32_t dst = ring + at * Cfg::kPair, bar = bars + at * 8;
      if (lacks) {
        kv4_bar_arrive(bar);
      } else {
        kv4_bar_expect(bar, x1 < 0 ? CB : 2 * CB);
        kv4_copy(dst, layer_pool + int64_t(x0) * CB, x1 == x0 + 1 ? 2 * CB : CB, bar);
        if (x1 >= 0 && x1 != x0 + 1) kv4_copy(dst + CB, layer_pool + int64_t(x1) * CB, CB, bar);
      }
    }
    issued++;
  };
#pragma unroll 1
  for (int i = 0; i < S; i++) issue();

  // O: dimensions 32 j + 4 gi + 2 z (+ 1: the last two) of tile 2 j + z; columns 2 tg, 2 tg + 1: heads 8 m + column, or
  // (N4) hi of heads 0..3, then lo
  float O[NT / 2][MT][4];
  uint32_t qa[N4 ? 1 : MT][HD / 16][N4 ? 2 : 4];
  // a lane's heads: gi (HB 8), gi and gi + 8 (HB 16), 2 (tg % 2) and the next one (N4)
  float mref[NH], l[NH], cs[NH];
  // The matrix products' sums lose a little towards 0 at each addition (131077 positions of 8 kv heads, 72 additions
  // a warp: 1.6e-6 of the result, where fp32 sums rounded to nearest are 0.7e-6 off), so every kFlush pairs they go,
  // rounded to nearest, to sums in shared memory, which stand in relation to the mref of then.  A pair is 4 additions
  // (N4: 2).  At 6 pairs the result is 0.8e-6 off and 0.6 us of 44 are spent on it, at 4 0.7e-6 and 1.1 us.
  // N4 holds hi + lo, the first half of the tiles with the lanes of hi, the others with those of lo.
  constexpr int kFlush = N4 ? 32 : 6, TILES = N4 ? NT / 4 : NT / 2;
  float4* acc = reinterpret_cast<float4*>(sm + Cfg::kAcc) + warp * (TILES * MT * 32) + lane;
  float* macc = reinterpret_cast<float*>(sm + Cfg::kLane) + warp * 64 + lane;   // [NH][32]
  int k = 0;                                  // pairs read
#pragma unroll 1
  while (k < count) {
    for (; pi0 < 0 && k < count; pi0++, k++) issue();
    if (k == count) break;
    // ---- a segment: consecutive pairs of one item
    const int seg = np - pi0 < count - k ? np - pi0 : count - k;
    int live = ent(e).y - pi0 * 2 * kKv4Chunk;   // positions from the pair on that exist
    bool poison = false;
    {
      // q of heads gi (and gi + 8; N4: gi % 4), split.  It is scaled by 8 log2(e) / sqrt(hd) (below 2) and a power of two that
      // brings a head's largest element into [2^10, 2^12), so that a score times cs, a power of two, is an exponent of 2 and
      // that product exact: the same number in the maximum and in the multiply-add of the weights, however large.  (With the
      // scale in cs, a maximum rounded by itself was off by up to half its last place: digits lost from scores of 2^26
      // on, the weight's whole range from 2^28.)
      const float* qb = a.q + int64_t(e) * a.q_stride + int64_t(g) * G * HD;
      float qx[MT][NG][8], back[MT];
#pragma unroll
      for (int m = 0; m < MT; m++) {
        const int h = N4 ? gi & 3 : gi + 8 * m;
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < NG; j++) {
          float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
          if (h < G) {
            u = *reinterpret_cast<const float4*>(qb + h * HD + 32 * j + 8 * tg);
            v = *reinterpret_cast<const float4*>(qb + h * HD + 32 * j + 8 * tg + 4);
          }
          qx[m][j][0] = u.x; qx[m][j][1] = u.y; qx[m][j][2] = u.z; qx[m][j][3] = u.w;
          qx[m][j][4] = v.x; qx[m][j][5] = v.y; qx[m][j][6] = v.z; qx[m][j][7] = v.w;
#pragma unroll
          for (int i = 0; i < 8; i++) top = fmaxf(top, fabsf(qx[m][j][i]));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int ex = int(__float_as_uint(top) >> 23);
        ex = ex < 14 ? 14 : ex;                                  // (zeros and values below 2^-113)
        const float up = __uint_as_float(uint32_t(264 - ex) << 23) * a.q_scale;   // 2^(137 - ex) q_scale
        back[m] = __uint_as_float(uint32_t(ex - 13) << 23);      // 2^(ex - 140)
#pragma unroll
        for (int j = 0; j < NG; j++)
#pragma unroll
          for (int i = 0; i < 8; i++) qx[m][j][i] *= up;
      }
#pragma unroll
      for (int j = 0; j < NG; j++)
#pragma unroll
        for (int i = 0; i < 4; i++) {   // pair (code i, code i + 4): k-step 2 j + i / 2, half i % 2
          const int kk = 2 * j + (i >> 1), r = i & 1;
          if constexpr (N4) {
            uint32_t hi, lo;
            kv4_split(qx[0][j][i], qx[0][j][i + 4], hi, lo);
            qa[0][kk][r] = gi < 4 ? hi : lo;
          } else if constexpr (MT == 1) {
            kv4_split(qx[0][j][i], qx[0][j][i + 4], qa[0][kk][2 * r], qa[0][kk][2 * r + 1]);
          } else {
            kv4_split(qx[0][j][i], qx[0][j][i + 4], qa[0][kk][2 * r], qa[MT - 1][kk][2 * r]);
            kv4_split(qx[MT - 1][j][i], qx[MT - 1][j][i + 4], qa[0][kk][2 * r + 1], qa[MT - 1][kk][2 * r + 1]);
          }
        }
#pragma unroll
      for (int m = 0; m < NH; m++) {
        cs[m] = N4 ? __shfl_sync(0xffffffffu, back[0], 4 * (2 * (tg & 1) + m)) : back[N4 ? 0 : m];
        mref[m] = -3e38f;
        l[m] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < NT / 2; i++)
#pragma unroll
        for (int m = 0; m < MT; m++) O[i][m][0] = O[i][m][1] = O[i][m][2] = O[i][m][3] = 0.f;
    }

    missing &= ~kHeld;
    const int kseg = k + seg;
#pragma unroll 1
    for (;;) {
#pragma unroll 1
    for (const int k1 = kseg - k < kFlush ? kseg : k + kFlush; k < k1; k++, live -= 2 * kKv4Chunk) {
      const int st = k & (S - 1);
      if (!(missing & kDead) &&
          !__all_sync(0xffffffffu, kv4_bar_wait(bars + st * 8, uint32_t(k / S) & 1u))) {
        missing |= kDead;
        if (lane == 0) kv4_flag(c, NT_KV4_TIMEOUT);
        for (int y = k; y < issued; y++)   // copies in flight land before anything else happens to the ring
          kv4_bar_wait(bars + (y & (S - 1)) * 8, uint32_t(y / S) & 1u);
      }
      if (missing & (kDead | (1u << st))) {
        poison = true;
        issue();
        continue;
      }
      const uint32_t base = ring + st * Cfg::kPair;

      // ---- scores of 32 positions
      float sc[4][4];
#pragma unroll
      for (int i = 0; i < 4; i++) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
      for (int u = 0; u < 2; u++) {
        uint32_t kw[2][NG], ks[2][NG / 2];
        float low[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};   // HB 16: the lo products' sums
#pragma unroll
        for (int i = 0; i < 2; i++) {
          kv4_words<NG>(base + u * CB + (i * 32 + lane) * (4 * NG), kw[i]);
          if (NG == 4) {
            const uint2 v = kv4_lds8(base + u * CB + L::kKS + (8 * i + gi) * (2 * NG));
            ks[i][0] = v.x; ks[i][NG / 2 - 1] = v.y;
          } else {
            ks[i][0] = kv4_lds4(base + u * CB + L::kKS + (8 * i + gi) * (2 * NG));
          }
        }
#pragma unroll
        for (int j = 0; j < NG; j++) {
          uint32_t b[2][4];
#pragma unroll
          for (int i = 0; i < 2; i++) {
            const uint32_t d = __byte_perm(ks[i][j >> 1], 0u, (j & 1) ? 0x3232u : 0x1010u);
            kv4_decode(kw[i][j], d, kv4_h2mul(d, kMinus72), b[i]);
          }
          // (products into the same accumulators never follow one another)
          if constexpr (N4) {   // 16 positions are the rows, the heads the columns; even and odd k-steps apart
#pragma unroll
            for (int y = 0; y < 2; y++) {
              const uint32_t w[4] = {b[0][2 * y], b[1][2 * y], b[0][2 * y + 1], b[1][2 * y + 1]};
              kv4_mma(sc[2 * u + y], w, qa[0][2 * j + y][0], qa[0][2 * j + y][1]);
            }
          } else {
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
              for (int y = 0; y < 2; y++)
#pragma unroll
                for (int i = 0; i < 2; i++)
                  kv4_mma(m ? low[i] : sc[2 * u + i], qa[m][2 * j + y], b[i][2 * y], b[i][2 * y + 1]);
          }
        }
        if constexpr (HB == 16) {
#pragma unroll
          for (int i = 0; i < 2; i++)
#pragma unroll
            for (int y = 0; y < 4; y++) sc[2 * u + i][y] += low[i][y];
        }
      }
      // the scores of this lane's heads; of the i-th this is the position
      auto at = [&](int i) { return N4 ? 16 * (i >> 1) + 8 * (i & 1) + gi : 8 * (i >> 1) + 2 * tg + (i & 1); };
      float x[NH][NX];
      if constexpr (N4) {
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
          for (int y = 0; y < 4; y++) {
            const float v = sc[2 * u][y] + sc[2 * u + 1][y];      // hi of columns tg < 2, lo of the others
            x[y & (NH - 1)][2 * u + (y >> 1)] = v + __shfl_xor_sync(0xffffffffu, v, 2);
          }
      } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int y = 0; y < 2; y++) {
            if (MT == 1) {
              x[0][(2 * i + y) % NX] = sc[i][y] + sc[i][y + 2];
            } else {
              x[0][(2 * i + y) % NX] = sc[i][y];
              x[NH - 1][(2 * i + y) % NX] = sc[i][y + 2];
            }
          }
      }
      if (live < 2 * kKv4Chunk) {
#pragma unroll
        for (int m = 0; m < NH; m++)
#pragma unroll
          for (int i = 0; i < NX; i++)
            if (at(i) >= live) x[m][i] = -INFINITY;
      }
      // ---- weights p = 2^(s - mref).  Only where a lane's sum passes 2^15 (at first it is infinite) is the maximum looked
      // for; where that passes mref by 12, as one of 8 weights does then, it less 6 becomes mref.  So weights stay within
      // f16, and the largest so far is at least 2^6: the lo terms of all that matter are ordinary f16 numbers.  (Exponents of
      // 2^25 and more are 4 or more apart, mref among them: the largest weight is 2^0 to 2^8 there, which serves as well.)
      float p[NH][NX], sum[NH];
      auto weights = [&]() {
#pragma unroll
        for (int m = 0; m < NH; m++) {
#pragma unroll
          for (int i = 0; i < NX; i++) p[m][i] = kv4_ex2(fmaf(x[m][i], cs[m], -mref[m]));
          sum[m] = (p[m][0] + p[m][1]) + (p[m][2] + p[m][3]);
          if constexpr (!N4) sum[m] += (p[m][4 % NX] + p[m][5 % NX]) + (p[m][6 % NX] + p[m][7 % NX]);
        }
      };
      weights();
      if (__any_sync(0xffffffffu, sum[0] > 32768.f || sum[NH - 1] > 32768.f)) {
        float f[NH];
#pragma unroll
        for (int m = 0; m < NH; m++) {
          float top = x[m][0];
#pragma unroll
          for (int i = 1; i < NX; i++) top = fmaxf(top, x[m][i]);
          top *= cs[m];
#pragma unroll
          for (int o = N4 ? 4 : 1; o <= (N4 ? 16 : 2); o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const float to = top - mref[m] > 12.f ? top - 6.f : mref[m];   // (mref + 12 could round past top)
          f[m] = kv4_ex2(mref[m] - to);
          mref[m] = to;
          l[m] *= f[m];
        }
#pragma unroll
        for (int m = 0; m < MT; m++) {
          const float f0 = N4 ? f[0] : __shfl_sync(0xffffffffu, f[m], 8 * tg);
          const float f1 = N4 ? f[NH - 1] : __shfl_sync(0xffffffffu, f[m], 8 * tg + 4);
#pragma unroll
          for (int i = 0; i < NT / 2; i++) {
            O[i][m][0] *= f0; O[i][m][1] *= f1;
            O[i][m][2] *= f0; O[i][m][3] *= f1;
          }
        }
        weights();
      }
#pragma unroll
      for (int m = 0; m < NH; m++) l[m] += sum[m];
      // P of chunk u as B operand: rows 2 tg, 2 tg + 1 (and + 8) are positions, column gi a head (+ 8 m)
      uint32_t hi[2][MT][2], lo[2][MT][2];   // (N4: hi holds both)
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int i = 0; i < 2; i++) {
          if constexpr (N4) {   // rows are positions, columns heads here: transposed
            uint32_t h2, l2;
            kv4_split(p[0][2 * u + i], p[NH - 1][2 * u + i], h2, l2);
            hi[u][0][i] = kv4_transpose(tg < 2 ? h2 : l2);
          } else {
#pragma unroll
            for (int m = 0; m < MT; m++)
              kv4_split(p[m][(4 * u + 2 * i) % NX], p[m][(4 * u + 2 * i + 1) % NX], hi[u][m][i], lo[u][m][i]);
          }
        }

      // ---- weighted values
#pragma unroll
      for (int u = 0; u < 2; u++) {
        uint32_t vw[2][NG], vs[2][NG];
#pragma unroll
        for (int r = 0; r < 2; r++) {
          kv4_words<NG>(base + u * CB + L::kV + (r * 32 + lane) * (4 * NG), vw[r]);
          kv4_words<NG>(base + u * CB + L::kVS + (r * 4 + tg) * (4 * NG), vs[r]);
        }
        if (u == 1) {
          __syncwarp();
          issue();   // the pair is in registers: its stage takes the next one
        }
        if (live < 2 * kKv4Chunk) {   // positions behind the end: scale 0, whatever the page holds there
#pragma unroll
          for (int r = 0; r < 2; r++) {
            const int v0 = 16 * u + 8 * r + 2 * tg;
            const uint32_t keep = (v0 < live ? 0xffffu : 0u) | (v0 + 1 < live ? 0xffff0000u : 0u);
#pragma unroll
            for (int j = 0; j < NG; j++) vs[r][j] &= keep;
          }
        }
#pragma unroll
        for (int j = 0; j < NG; j++) {
          uint32_t b[2][4];
#pragma unroll
          for (int r = 0; r < 2; r++) kv4_decode(vw[r][j], vs[r][j], kv4_h2mul(vs[r][j], kMinus72), b[r]);
#pragma unroll
          for (int m = 0; m < MT; m++)
#pragma unroll
            for (int z = 0; z < 2; z++) {
              const uint32_t v[4] = {b[0][2 * z], b[0][2 * z + 1], b[1][2 * z], b[1][2 * z + 1]};
              kv4_mma(O[2 * j + z][m], v, hi[u][m][0], hi[u][m][1]);
            }
          if constexpr (!N4) {
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
              for (int z = 0; z < 2; z++) {
                const uint32_t v[4] = {b[0][2 * z], b[0][2 * z + 1], b[1][2 * z], b[1][2 * z + 1]};
                kv4_mma(O[2 * j + z][m], v, lo[u][m][0], lo[u][m][1]);
              }
          }
        }
      }
    }

      // O, and what is held if anything is, to the sums; or, at the segment's end, into O
      const bool last = k == kseg, held = missing & kHeld;
      if (last && !held) break;
#pragma unroll
      for (int m = 0; m < MT; m++) {
        float f0 = 0.f, f1 = 0.f;   // of the sums: 2^(their mref - mref)
        if (held) {
          const float f = kv4_ex2(macc[32 * m] - mref[m]);
          f0 = N4 ? f : __shfl_sync(0xffffffffu, f, 8 * tg);
          f1 = N4 ? kv4_ex2(macc[32 * (NH - 1)] - mref[NH - 1]) : __shfl_sync(0xffffffffu, f, 8 * tg + 4);
        }
#pragma unroll
        for (int i = 0; i < TILES; i++) {   // (N4: tile i of the lanes of hi, TILES + i of those of lo)
          float4* y = acc + (i * MT + m) * 32;
          const bool second = N4 && tg >= 2;
          float o[4];
#pragma unroll
          for (int x = 0; x < 4; x++) {
            o[x] = second ? O[(i + TILES) % (NT / 2)][m][x] : O[i][m][x];
            if (N4 && !last) o[x] += __shfl_xor_sync(0xffffffffu, second ? O[i][m][x] : O[(i + TILES) % (NT / 2)][m][x], 2);
          }
          if (held) {
            const float4 v = *y;
            o[0] = fmaf(v.x, f0, o[0]); o[1] = fmaf(v.y, f1, o[1]);
            o[2] = fmaf(v.z, f0, o[2]); o[3] = fmaf(v.w, f1, o[3]);
          }
          if (!last) *y = make_float4(o[0], o[1], o[2], o[3]);
#pragma unroll
          for (int x = 0; x < 4; x++) {
            if (!second) O[i][m][x] = last ? o[x] : 0.f;
            if (N4 && (second || !last)) O[(i + TILES) % (NT / 2)][m][x] = last ? o[x] : 0.f;
            if (N4 && second && !last) O[i][m][x] = 0.f;
          }
        }
      }
      if (last) break;
#pragma unroll
      for (int m = 0; m < NH; m++) macc[32 * m] = mref[m];
      missing |= kHeld;
    }

    // ---- the end of the segment
#pragma unroll
    for (int m = 0; m < NH; m++) {
#pragma unroll
      for (int o = N4 ? 4 : 1; o <= (N4 ? 16 : 2); o <<= 1) l[m] += __shfl_xor_sync(0xffffffffu, l[m], o);
      if (poison) l[m] = NAN;
    }
    const bool whole = pi0 == 0 && seg == np;
    const int slot = 2 * warp + (pi0 > 0 ? 0 : 1), e_was = e, g_was = g;
    if (k < count) locate(w0 + k, e, g, pi0, np);
    float* po = slot_ptr(slot);
    if (!whole && lane == 0) slot_item[slot] = e_was * c.n_kv + g_was;
    __syncwarp();   // (slot 1 is the ring: every lane has read its last pair)
    float* to = whole ? a.out + int64_t(e_was) * a.out_stride + int64_t(g_was) * G * HD : po;
    if constexpr (N4) {   // lanes tg < 2 store head 2 (tg % 2), the others the next one, dimensions 32 j + 4 gi + 0..3
      const int y = tg >> 1, h = 2 * (tg & 1) + y;
      const float f = whole ? 1.f / (y ? l[NH - 1] : l[0]) : 1.f;
      if (!whole && gi == 0) reinterpret_cast<float2*>(po + ROWS * HD)[h] = make_float2(y ? mref[NH - 1] : mref[0], y ? l[NH - 1] : l[0]);
#pragma unroll
      for (int j = 0; j < NG; j++) {
        float o[2][4];
#pragma unroll
        for (int z = 0; z < 2; z++)
#pragma unroll
          for (int i = 0; i < 4; i++) {   // hi + lo
            const float v = O[2 * j + z][0][i];
            o[z][i] = v + __shfl_xor_sync(0xffffffffu, v, 2);
          }
        if (h < G)
          *reinterpret_cast<float4*>(to + h * HD + 32 * j + 4 * gi) =
              make_float4((y ? o[0][1] : o[0][0]) * f, (y ? o[0][3] : o[0][2]) * f, (y ? o[1][1] : o[1][0]) * f,
                          (y ? o[1][3] : o[1][2]) * f);
      }
    } else {
#pragma unroll
      for (int m = 0; m < MT; m++) {
        if (!whole && tg == 0) reinterpret_cast<float2*>(po + ROWS * HD)[gi + 8 * m] = make_float2(mref[m], l[m]);
#pragma unroll
        for (int y = 0; y < 2; y++) {   // head 8 m + 2 tg + y: dimensions 32 j + 4 gi + 0..3
          const int h = 8 * m + 2 * tg + y;
          const float lh = __shfl_sync(0xffffffffu, l[m], 8 * tg + 4 * y), f = whole ? 1.f / lh : 1.f;
          if (h < G) {
#pragma unroll
            for (int j = 0; j < NG; j++)
              *reinterpret_cast<float4*>(to + h * HD + 32 * j + 4 * gi) =
                  make_float4(O[2 * j][m][y] * f, O[2 * j][m][y + 2] * f, O[2 * j + 1][m][y] * f, O[2 * j + 1][m][y + 2] * f);
          }
        }
      }
    }
  }

  // ---- merge within the CTA: a warp per head, a lane per slot; an item's slots in order
  if (CL && total <= share) return;   // one warp has done it all (the whole cluster knows)
  __syncthreads();
  constexpr int V = HD / 32;
  kv4_merge<HD, ROWS, NW, 2 * NW>(
      c, a, slot_item, slot_ptr, reinterpret_cast<int*>(sm + Cfg::kLane) + warp * 64,
      [&](int item, int& first, int& units) {
        const int ie = item / c.n_kv;
        units = kv4_pairs(ent(ie).y);
        first = CL ? 0 : prefix[ie] + item % c.n_kv * (units + kKv4ItemPairs) + kKv4ItemPairs;
      },
      c0, c1, NW * share, part0, CL ? nullptr : header);

  // ---- CL: merge across the cluster, a warp per head
  if constexpr (CL) {
    if (total <= NW * share) return;   // the first CTA has had it all, and written it (the whole cluster knows)
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    const int ranks = (total + NW * share - 1) / (NW * share);   // CTAs that had pairs
    for (int h = int(blockIdx.x) * NW + warp; h < G; h += int(gridDim.x) * NW) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < ranks) ml = reinterpret_cast<const float2*>(cl.map_shared_rank(part0, unsigned(lane)) + ROWS * HD)[h];
      float M = ml.x;
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      float f = lane < ranks ? kv4_ex2(ml.x - M) : 0.f, sum = ml.y * f;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      f /= sum;
      float o[V];
#pragma unroll
      for (int v = 0; v < V; v++) o[v] = 0.f;
#pragma unroll 4
      for (int b = 0; b < ranks; b++) {
        const float fb = __shfl_sync(0xffffffffu, f, b);
        const float* r = cl.map_shared_rank(part0, unsigned(b)) + h * HD + V * lane;
        if (V == 4) {
          const float4 x = *reinterpret_cast<const float4*>(r);
          o[0] = fmaf(x.x, fb, o[0]); o[1] = fmaf(x.y, fb, o[1]);
          o[2 % V] = fmaf(x.z, fb, o[2 % V]); o[3 % V] = fmaf(x.w, fb, o[3 % V]);
        } else {
          const float2 x = *reinterpret_cast<const float2*>(r);
          o[0] = fmaf(x.x, fb, o[0]); o[1] = fmaf(x.y, fb, o[1]);
        }
      }
      float* to = a.out + int64_t(e_own) * a.out_stride + (int64_t(g_own) * G + h) * HD + V * lane;
      if (V == 4) *reinterpret_cast<float4*>(to) = make_float4(o[0], o[1], o[2 % V], o[3 % V]);
      else *reinterpret_cast<float2*>(to) = make_float2(o[0], o[1]);
    }
    cl.sync();   // the partial results stay until every CTA has read them
  }
}

// Items that several CTAs worked on: CTA (b, h) merges query head h of the item that
// CTA b of k_kv4_attn began and others ended.  A warp reads a row of partial
// results per step, the warps' sums are added in order.
constexpr int kKv4MergeWarps = 8;
template <int HD>
__global__ void __launch_bounds__(32 * kKv4MergeWarps) k_kv4_attn_merge(Kv4 c, Kv4AttnArgs a, int part_floats, int rows) {
  constexpr int V = HD / 32;
  __shared__ float s_o[kKv4MergeWarps][HD];
  __shared__ float2 s_ml[kKv4MergeWarps];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, h = blockIdx.y;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float* first = a.part + (int64_t(blockIdx.x) * 2 + 1) * part_floats;   // slot 1, then slot 0 of the next CTAs
  const int2 header = __ldcg(reinterpret_cast<const int2*>(first + part_floats - 4));
  const int most = int(gridDim.x + 1 - blockIdx.x);   // CTAs from this one on
  // a warp takes members warp, warp + 8, ...; the first three are read beside the header, before it is known who they are
  float M = -INFINITY, sum = 0.f, o[V];
#pragma unroll
  for (int v = 0; v < V; v++) o[v] = 0.f;
  int members = most;
  for (int b0 = warp; b0 < members; b0 += 3 * kKv4MergeWarps) {
    float2 ml[3];
    float x[3][V];
#pragma unroll
    for (int u = 0; u < 3; u++) {
      const int b = b0 + u * kKv4MergeWarps;
      if (b < members) {
        const float* r = b ? first + (int64_t(b) * 2 - 1) * part_floats : first;
        ml[u] = __ldcg(reinterpret_cast<const float2*>(r + rows * HD) + h);
        if (V == 4) {
          const float4 y = __ldcg(reinterpret_cast<const float4*>(r + h * HD) + lane);
          x[u][0] = y.x; x[u][1] = y.y; x[u][2 % V] = y.z; x[u][3 % V] = y.w;
        } else {
          const float2 y = __ldcg(reinterpret_cast<const float2*>(r + h * HD) + lane);
          x[u][0] = y.x; x[u][1] = y.y;
        }
      }
    }
    if (header.x < 0) return;   // (the whole CTA: no barrier has been passed)
    members = header.y;
#pragma unroll
    for (int u = 0; u < 3; u++) {
      if (b0 + u * kKv4MergeWarps >= members) continue;
      const float to = fmaxf(M, ml[u].x), was = kv4_ex2(M - to), f = kv4_ex2(ml[u].x - to);
      M = to;
      sum = fmaf(sum, was, ml[u].y * f);
#pragma unroll
      for (int v = 0; v < V; v++) o[v] = fmaf(o[v], was, x[u][v] * f);
    }
  }
  if (header.x < 0) return;
#pragma unroll
  for (int v = 0; v < V; v++) s_o[warp][lane * V + v] = o[v];
  if (lane == 0) s_ml[warp] = make_float2(M, sum);
  __syncthreads();
  if (t < HD) {
    float top = -INFINITY, total = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kKv4MergeWarps; w++) top = fmaxf(top, s_ml[w].x);
#pragma unroll
    for (int w = 0; w < kKv4MergeWarps; w++) {
      const float f = kv4_ex2(s_ml[w].x - top);
      total = fmaf(s_ml[w].y, f, total);
      y = fmaf(s_o[w][t], f, y);
    }
    const int e = header.x / c.n_kv, g = header.x % c.n_kv;
    a.out[int64_t(e) * a.out_stride + (int64_t(g) * a.G + h) * HD + t] = y / total;
  }
}

// CTAs of a cluster, and how many such clusters of the attention kernel the GPU
// holds at once (0: none).
constexpr int kKv4Clusters[6] = {1, 2, 4, 8, 12, 16};
struct Kv4Fit {
  KernelSetup setup;
  int clusters[6] = {0, 0, 0, 0, 0, 0};
};
static void kv4_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], dim3 grid, int threads, size_t smem,
                       cudaStream_t s, int cluster) {
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
static Kv4Fit kv4_fit() {
  using Cfg = Kv4AttnCfg<HD, HB>;
  Kv4Fit f;
  f.setup = kernel_setup(k_kv4_attn<HD, HB, true>, Cfg::kSmem);
  if (f.setup.err == cudaSuccess)
    f.setup.err = cudaFuncSetAttribute(k_kv4_attn<HD, HB, true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  for (int i = 0; i < 6 && f.setup.err == cudaSuccess; i++) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    kv4_config(cfg, attr, dim3(unsigned(kKv4Clusters[i])), Cfg::kThreads, Cfg::kSmem, nullptr, kKv4Clusters[i]);
    cfg.numAttrs = 1;
    attr[0] = attr[1];
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, k_kv4_attn<HD, HB, true>, &cfg) == cudaSuccess) f.clusters[i] = n;
    else cudaGetLastError();   // (no such cluster: it is not taken)
  }
  return f;
}

// Most pairs of a warp in the form with a cluster per item.  (us, that form with up to 2
// pairs, with up to 3, and the other: 1 sequence of 4161 positions, 64/8 heads: 9.6,
// 9.6, 10.4; of 600: 8.1, 8.1, 9.9; 16 of 300, 32/8: 6.8, 6.8, 11.0; 1 of 9000, 16/1: 11.4, 14.7, 11.4.)
constexpr int kKv4ClusterShare = 2;

// Tiles of 128 positions an SM, by capacity, from which the tcgen05 kernel is taken (8 and 16 heads of 128 dimensions; below,
// its tiles are too coarse a share).  (us, this file's kernel and that one: 1 sequence of 9000, 16/1 heads, 0.5 tiles
// an SM: 11.4, 13.1; of 70000: 3.6: 17.3, 18.2; 1 of 12000, 64/8: 4.9: 13.1, 13.8; 1 of 16000: 6.6: 15.0, 14.0.)
constexpr int kKv4TcTiles = 6;

// Pairs of an item's capacity per warp of a CTA up to which CTAs take whole items: no second launch, a CTA's share uneven
// by an item.  (us, whole and cut: 30 sequences of 300, 64/8 heads: 11.1, 13.0; 25 of 150: 9.4, 11.7; 100 of 90: 14.7,
// 17.0; 64 of up to 200, 32/8: 14.0, 14.3; of 200, 64/8: 13.8, 13.5; at 2 pairs 20 of 700, 64/8: 14.8, 15.6, and 64 of 700,
// 32/8: 22.6, 24.1; at 5 30 of up to 2500, 32/8: 28.7, 22.9.)
constexpr int kKv4WholeShare = 2;

template <int HD, int HB>
static cudaError_t kv4_launch_attn(const Kv4& k, const Kv4AttnArgs& a, int64_t most_units, cudaStream_t s) {
  using Cfg = Kv4AttnCfg<HD, HB>;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  // A cluster per item where all of them fit the GPU at once and their capacity leaves no warp more than kKv4ClusterShare
  // pairs: the smallest such that a warp has one pair at most, or the largest.
  static const Kv4Fit fit = kv4_fit<HD, HB>();
  if (fit.setup.err != cudaSuccess) return fit.setup.err;
  const int64_t items = int64_t(a.n) * k.n_kv, pairs = (int64_t(k.max_pages) * k.page_len + 31) / 32;
  int cluster = 0;
  for (int i = 0; i < 6; i++) {
    if (fit.clusters[i] < items || pairs > int64_t(kKv4Clusters[i]) * Cfg::NW * kKv4ClusterShare) continue;
    cluster = kKv4Clusters[i];
    if (pairs <= int64_t(cluster) * Cfg::NW) break;
  }
  if (cluster) {
    kv4_config(cfg, attr, dim3(unsigned(cluster), unsigned(items)), Cfg::kThreads, Cfg::kSmem, s, cluster);
    return cudaLaunchKernelEx(&cfg, k_kv4_attn<HD, HB, true>, k, a);
  }
  int ctas = 0;
  cudaError_t e = cudaSuccess;
  // Whole items for the CTAs where each is small: nothing is left to a second launch.
  const bool whole = pairs <= int64_t(Cfg::NW) * kKv4WholeShare;
  bool tc = false;
  if constexpr (HD == 128 && HB >= 8) {
    tc = !whole && items * ((pairs + 3) / 4) >= int64_t(kKv4TcTiles) * fit.setup.sms && kv4_attn_tc_runs(a.G);
    if (tc) e = kv4_launch_attn_tc(k, a, s, &ctas);
  }
  if (!tc) {
    const auto kernel = whole ? k_kv4_attn<HD, HB, false, true> : k_kv4_attn<HD, HB, false>;
    static const KernelSetup setups[2] = {kernel_setup(k_kv4_attn<HD, HB, false>, Cfg::kSmem),
                                          kernel_setup(k_kv4_attn<HD, HB, false, true>, Cfg::kSmem)};
    const KernelSetup& setup = setups[whole];
    if (setup.err != cudaSuccess) return setup.err;
    const int64_t useful = (most_units + Cfg::NW * kKv4MinPairs - 1) / (Cfg::NW * kKv4MinPairs);
    ctas = setup.sms < kKv4AttnMaxCtas ? setup.sms : kKv4AttnMaxCtas;
    if (ctas > useful) ctas = int(useful);
    kv4_config(cfg, attr, dim3(unsigned(ctas)), Cfg::kThreads, Cfg::kSmem, s, 0);
    e = cudaLaunchKernelEx(&cfg, kernel, k, a);
  }
  if (e != cudaSuccess || ctas < 2 || whole) return e;
  // (the last CTA's items end with it)
  kv4_config(cfg, attr, dim3(unsigned(ctas - 1), unsigned(a.G)), 32 * kKv4MergeWarps, 0, s, 0);
  return cudaLaunchKernelEx(&cfg, k_kv4_attn_merge<HD>, k, a, int(Cfg::kPart), int(Cfg::kRows));
}

}  // namespace nt

using namespace nt;

extern "C" nt_status nt_attention_kv4(const nt_kv4_cache* c, int32_t layer, int32_t n_heads, int32_t n,
                                      const int32_t* dev_seq, const float* dev_q, int64_t q_stride, float* dev_out,
                                      int64_t out_stride, void* dev_workspace, size_t workspace_bytes, void* stream) {
  Kv4 k;
  nt_status st = kv4_check(c, "nt_attention_kv4", true, &k);
  if (st) return st;
  auto bad = [](const char* what) { return fail(NT_E_INVAL, std::string("nt_attention_kv4: ") + what); };
  if (layer < 0 || layer >= k.n_layers) return bad("layer out of range");
  if (n_heads < 1 || n_heads % k.n_kv) return bad("n_heads must be a positive multiple of n_kv_heads");
  const int G = n_heads / k.n_kv;
  if (G != 1 && G != 2 && G != 4 && G != 8 && G != 16)
    return fail(NT_E_UNSUPPORTED, "nt_attention_kv4: query heads per kv head must be 1, 2, 4, 8 or 16");
  if (int64_t(k.n_pages) * k.n_kv * (k.page_len / kKv4Chunk) > 0x7fffffffLL) return bad("a layer of the pool has more than 2^31 - 1 chunks");
  if (n_heads > 65535) return bad("n_heads above 65535");
  if (n < 0 || n > 65536 || (!dev_seq && n > k.max_seqs)) return bad("n out of range");
  const int64_t row = int64_t(n_heads) * k.hd;
  if (q_stride < row || out_stride < row || q_stride % 4 || out_stride % 4 || q_stride > (int64_t(1) << 40) ||
      out_stride > (int64_t(1) << 40))
    return bad("strides must be multiples of 4 and at least n_heads * head_dim");
  if (!kv4_aligned(dev_q, 16) || !kv4_aligned(dev_out, 16) || !kv4_aligned(dev_workspace, 16))
    return bad("q, out or workspace is NULL or not 16-byte aligned");
  if (dev_seq && !kv4_aligned(dev_seq, 4)) return bad("seq is not 4-byte aligned");
  const size_t wb = kv4_attn_ws_bytes(n_heads, k.n_kv, k.hd);
  if (workspace_bytes < wb) return bad("workspace too small");
  if (n == 0) return NT_OK;
  const int64_t qb = ((n - 1) * q_stride + row) * 4, ob = ((n - 1) * out_stride + row) * 4;
  if (kv4_overlap(dev_out, ob, dev_q, qb) || kv4_overlap(dev_out, ob, dev_workspace, int64_t(wb)) ||
      kv4_overlap(dev_q, qb, dev_workspace, int64_t(wb)) || kv4_meets_cache(k, dev_out, ob) ||
      kv4_meets_cache(k, dev_workspace, int64_t(wb)) ||
      (dev_seq && (kv4_overlap(dev_seq, int64_t(n) * 4, dev_out, ob) ||
                   kv4_overlap(dev_seq, int64_t(n) * 4, dev_workspace, int64_t(wb)))))
    return bad("the output or the workspace overlaps another buffer");
  Kv4AttnArgs a{};
  a.layer = layer;
  a.G = G;
  a.q_scale = 11.541560327111707f / sqrtf(float(k.hd));
  a.part = static_cast<float*>(dev_workspace);
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  const int64_t entry_pairs = int64_t(k.n_kv) * ((int64_t(k.max_pages) * k.page_len + 31) / 32 + kKv4ItemPairs);
  // a launch's pairs are counted in 32 bits
  const int64_t most = int64_t(1) << 30;
  if (entry_pairs > most) return bad("n_kv_heads * max_pages * page_len is too large");
  const int32_t batch = entry_pairs * kKv4Batch <= most ? kKv4Batch : int32_t(most / entry_pairs);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int32_t i = 0; i < n; i += batch) {
    a.n = n - i < batch ? n - i : batch;
    a.seq0 = i;
    a.seq = dev_seq ? dev_seq + i : nullptr;
    a.q = dev_q + int64_t(i) * q_stride;
    a.out = dev_out + int64_t(i) * out_stride;
    cudaError_t e;
    const int64_t units = a.n * entry_pairs;
    if (k.hd == 64)
      e = G <= 4 ? kv4_launch_attn<64, 4>(k, a, units, s)
                 : (G == 8 ? kv4_launch_attn<64, 8>(k, a, units, s) : kv4_launch_attn<64, 16>(k, a, units, s));
    else
      e = G <= 4 ? kv4_launch_attn<128, 4>(k, a, units, s)
                 : (G == 8 ? kv4_launch_attn<128, 8>(k, a, units, s) : kv4_launch_attn<128, 16>(k, a, units, s));
    if (e != cudaSuccess) return cuda_fail(e, "nt_attention_kv4");
  }
  return NT_OK;
}
