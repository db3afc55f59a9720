// nt_kv4_attn.cu -- GQA decode attention over the paged 4-bit K/V cache.
#include "nt_kv4.cuh"

namespace nt {

size_t kv4_attn_ws_bytes(int, int, int) { return 16; }

struct Kv4AttnArgs {
  int32_t layer, n_heads, n;
  const int32_t* seq;
  const float* q;
  int64_t q_stride;
  float* out;
  int64_t out_stride;
};

// One CTA per (sequence, kv head): chunks of 16 positions are dequantized into
// shared memory, scored against the G query heads, and folded into the running
// maximum, sum and output of each head.
template <int HD>
__global__ void __launch_bounds__(256) k_kv4_attn(Kv4 c, Kv4AttnArgs a, int G, float scale) {
  using L = Kv4Chunk<HD>;
  __shared__ float q[16 * HD], ks[16][HD], vs[16][HD], ps[16][16], corr[16], ml[16][2];
  const int i = blockIdx.x, g = blockIdx.y, t = threadIdx.x;
  const int s = a.seq ? a.seq[i] : i;
  const float* qi = a.q + int64_t(i) * a.q_stride + int64_t(g) * G * HD;
  float* oi = a.out + int64_t(i) * a.out_stride + int64_t(g) * G * HD;
  const bool bad_seq = s < 0 || s >= c.max_seqs;
  const int len = bad_seq ? 0 : c.len[s];
  bool poison = bad_seq || len < 0 || len > c.capacity();
  if (poison && t == 0) kv4_flag(c, bad_seq ? NT_KV4_BAD_SEQ : NT_KV4_BAD_LEN);
  for (int e = t; e < G * HD; e += 256) q[e] = qi[e];
  if (t < G) { ml[t][0] = -INFINITY; ml[t][1] = 0.f; }
  float acc[16 * HD / 256];
#pragma unroll
  for (int e = 0; e < 16 * HD / 256; e++) acc[e] = 0.f;
  for (int t0 = 0; t0 < len && !poison; t0 += 16) {
    const int page = c.table[int64_t(s) * c.max_pages + t0 / c.page_len], live = min(16, len - t0);
    if (page < 0 || page >= c.n_pages) {   // uniform over the CTA
      poison = true;
      if (t == 0) kv4_flag(c, NT_KV4_BAD_PAGE);
      break;
    }
    const uint8_t* ch = c.chunk(a.layer, page, g, t0 % c.page_len);
    __syncthreads();
    for (int e = t; e < 16 * HD; e += 256) {
      const int p = e / HD, d = e % HD, j = d / 32;
      if (p < live) {
        const uint32_t kw = *reinterpret_cast<const uint32_t*>(ch + L::k_word(p, d / 8 % 4, j));
        const uint32_t vh = *reinterpret_cast<const uint16_t*>(ch + L::v_half(p, d / 4 % 8, j));
        ks[p][d] = __half2float(*reinterpret_cast<const __half*>(ch + L::k_scale(p, j))) * float(int(kw >> (4 * (d % 8)) & 15u) - 8);
        vs[p][d] = __half2float(*reinterpret_cast<const __half*>(ch + L::v_scale(p, j))) * float(int(vh >> (4 * (d % 4)) & 15u) - 8);
      } else {
        ks[p][d] = vs[p][d] = 0.f;
      }
    }
    __syncthreads();
    if (t < 16 * G) {
      float x = 0.f;
      for (int d = 0; d < HD; d++) x = fmaf(q[(t / 16) * HD + d], ks[t % 16][d], x);
      ps[t / 16][t % 16] = t % 16 < live ? x * scale : -INFINITY;
    }
    __syncthreads();
    if (t < G) {
      float m = ml[t][0];
      for (int p = 0; p < 16; p++) m = fmaxf(m, ps[t][p]);
      const float w = expf(ml[t][0] - m);
      float l = ml[t][1] * w;
      for (int p = 0; p < 16; p++) l += (ps[t][p] = expf(ps[t][p] - m));
      corr[t] = w;
      ml[t][0] = m;
      ml[t][1] = l;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 16 * HD / 256; e++) {
      const int h = (t + 256 * e) / HD, d = (t + 256 * e) % HD;
      if (h < G) {
        acc[e] *= corr[h];
        for (int p = 0; p < 16; p++) acc[e] = fmaf(ps[h][p], vs[p][d], acc[e]);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 16 * HD / 256; e++) {
    const int h = (t + 256 * e) / HD, d = (t + 256 * e) % HD;
    if (h < G) oi[h * HD + d] = poison ? NAN : (len ? acc[e] / ml[h][1] : 0.f);
  }
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
  const Kv4AttnArgs a{layer, n_heads, n, dev_seq, dev_q, q_stride, dev_out, out_stride};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid{unsigned(n), unsigned(k.n_kv)};
  const float scale = 1.0f / sqrtf(float(k.hd));
  if (k.hd == 64) k_kv4_attn<64><<<grid, 256, 0, s>>>(k, a, G, scale);
  else k_kv4_attn<128><<<grid, 256, 0, s>>>(k, a, G, scale);
  NT_CUDA(cudaGetLastError());
  return NT_OK;
}
