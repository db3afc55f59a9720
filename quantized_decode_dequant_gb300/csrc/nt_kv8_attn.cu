// nt_kv8_attn.cu -- attention over the paged 8-bit cache (include/nt.h,
// nt_attention_kv8).
#include "nt_kv8.cuh"

namespace nt {

struct Kv8AttnArgs {
  int32_t layer, n, G, k;
  const int32_t* seq;
  const int32_t* ctx;
  const int32_t* pages;
  const float* q;
  int64_t q_stride;
  float* out;
  int64_t out_stride;
  float scale;          // log2(e) / sqrt(hd)
};

size_t kv8_attn_ws_bytes(int n_heads, int n_kv, int hd) { return 16; }

// A CTA per (entry, kv head), a warp per query head: 32 positions at a time, a lane's
// score that of its position, then a lane's sums those of its dimensions.
template <int HD>
__global__ void __launch_bounds__(256) k_kv8_attn(Kv4 c, Kv8AttnArgs a) {
  constexpr int V = HD / 32;
  __shared__ float s_q[kKv8MaxGroup * HD];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int i = int(blockIdx.x / c.n_kv), g = int(blockIdx.x % c.n_kv);
  kv4_dependent();
  const int s = a.seq ? a.seq[i] : i;
  float* out = a.out + int64_t(i) * a.out_stride + int64_t(g) * a.G * HD;
  uint32_t bad = 0;
  int n = 0;
  if (s < 0 || s >= c.max_seqs) {
    bad = NT_KV4_BAD_SEQ;
  } else {
    const int len = c.len[s];
    n = a.ctx ? a.ctx[i] : len;
    if (len < 0 || len > c.capacity() || n < 0 || n > len) bad = NT_KV4_BAD_LEN;
  }
  if (bad || n == 0) {
    if (bad && t == 0) kv4_flag(c, bad);
    for (int x = t; x < a.G * HD; x += 256) out[x] = bad ? NAN : 0.f;
    return;
  }
  for (int x = t; x < a.G * HD; x += 256) s_q[x] = a.q[int64_t(i) * a.q_stride + int64_t(g) * a.G * HD + x];
  __syncthreads();
  const int m = int((int64_t(n) + c.page_len - 1) / c.page_len), count = a.k ? a.k : m;
  const int32_t* list = a.k ? a.pages + (int64_t(i) * c.n_kv + g) * a.k : nullptr;
  const Kv8Page L(c);
  for (int h = warp; h < a.G; h += 8) {
    float M = -INFINITY, sum = 0.f, o[V];
    bool nan = false;
    int seen = 0, before = -1;
#pragma unroll
    for (int v = 0; v < V; v++) o[v] = 0.f;
    for (int x = 0; x < count; x++) {
      const int j = list ? list[x] : x;
      if (j < 0) break;
      const int page = j < m && j > before ? c.table[int64_t(s) * c.max_pages + j] : -1;
      before = j;
      if (page < 0 || page >= c.n_pages) {
        if (lane == 0) kv4_flag(c, NT_KV4_BAD_PAGE);
        nan = true;
        break;
      }
      const uint8_t* base = c.pool + (int64_t(a.layer) * c.n_pages + page) * c.page_bytes();
      const int8_t* ex = reinterpret_cast<const int8_t*>(base + L.exps(g));
      const float fk = kv8_exp2i(ex[0]), fv = kv8_exp2i(ex[1]);
      const int live = n - j * c.page_len < c.page_len ? n - j * c.page_len : c.page_len;
      for (int p0 = 0; p0 < live; p0 += 32) {
        const int p = p0 + lane;
        float y = -INFINITY;
        if (p < live) {
          y = 0.f;
          for (int ch = 0; ch < HD / 16; ch++) {
            const uint4 w = *reinterpret_cast<const uint4*>(base + L.k(g) + kv8_k_at(HD, p, ch));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int d = 0; d < 8; d++) {
              const float2 z = kv8_value2(u[d >> 1] >> (16 * (d & 1)));
              y = fmaf(z.x, s_q[h * HD + 16 * ch + 2 * d], y);
              y = fmaf(z.y, s_q[h * HD + 16 * ch + 2 * d + 1], y);
            }
          }
          y = y * fk * a.scale;
          nan |= y != y;
        }
        float top = y;
#pragma unroll
        for (int b = 16; b; b >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, b));
        const float to = fmaxf(M, top), f = exp2f(M - to), w = p < live ? exp2f(y - to) : 0.f;
        M = to;
        sum = sum * f + w;
#pragma unroll
        for (int v = 0; v < V; v++) o[v] *= f;
        for (int tc = p0 / 16; tc * 16 < live && tc < p0 / 16 + 2; tc++)
#pragma unroll
          for (int v = 0; v < V; v++) {
            const uint4 z = *reinterpret_cast<const uint4*>(base + L.v(g) + kv8_v_at(HD, tc, 32 * v + lane));
            const uint32_t u[4] = {z.x, z.y, z.z, z.w};
            for (int b = 0; b < 16; b++) {
              if (tc * 16 + b >= live) break;
              const float2 r = kv8_value2(u[b >> 2] >> (16 * (b >> 1 & 1)));
              o[v] = fmaf((b & 1 ? r.y : r.x) * fv, __shfl_sync(0xffffffffu, w, tc * 16 - p0 + b), o[v]);
            }
          }
      }
      seen += live;
    }
    nan = __any_sync(0xffffffffu, nan);
#pragma unroll
    for (int b = 16; b; b >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, b);
#pragma unroll
    for (int v = 0; v < V; v++) out[h * HD + 32 * v + lane] = nan ? NAN : seen ? o[v] / sum : 0.f;
  }
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
  if (n_heads / k.n_kv > kKv8MaxGroup) return fail(NT_E_UNSUPPORTED, std::string(who) + ": more than 16 query heads per kv head");
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
  const size_t wb = kv8_attn_ws_bytes(n_heads, k.n_kv, k.hd);
  if (workspace_bytes < wb) return bad("workspace too small");
  const int64_t items = int64_t(n) * k.n_kv;
  if (items > (1 << 24)) return bad("n * n_kv_heads above 2^24");
  if (n == 0) return NT_OK;
  const int64_t qb = ((n - 1) * q_stride + row) * 4, ob = ((n - 1) * out_stride + row) * 4, lb = int64_t(n) * 4;
  auto meets = [&](const void* p, int64_t bytes) {   // a written buffer and everything else
    return kv4_meets_cache(k, p, bytes) || kv4_overlap(p, bytes, dev_q, qb) || (dev_seq && kv4_overlap(p, bytes, dev_seq, lb)) ||
           (dev_ctx && kv4_overlap(p, bytes, dev_ctx, lb)) || (n_select && kv4_overlap(p, bytes, dev_pages, items * n_select * 4));
  };
  if (meets(dev_out, ob) || meets(dev_workspace, int64_t(wb)) || kv4_overlap(dev_out, ob, dev_workspace, int64_t(wb)))
    return bad("the output or the workspace overlaps another buffer");
  const Kv8AttnArgs a{layer, n, n_heads / k.n_kv, n_select, dev_seq, dev_ctx, dev_pages, dev_q, q_stride, dev_out, out_stride,
                      1.4426950408889634f / sqrtf(float(k.hd))};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  NT_CUDA(k.hd == 64 ? kv4_launch(k_kv8_attn<64>, unsigned(items), 256u, s, k, a) : kv4_launch(k_kv8_attn<128>, unsigned(items), 256u, s, k, a));
  return NT_OK;
}
