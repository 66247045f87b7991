// Multi-query paged attention over quantized KV caches (E4M3 and 4-bit pools):
// chunks of new tokens, single tokens among them, causal, with an optional
// sliding window.
//
// What it computes, with K and V the values the codes stand for before the
// tensor's scale, for the new token at position p of its sequence:
//   s_t = scale * k_scale * q . K_t,  o = v_scale * sum_t softmax(s)_t V_t,
// t over [max(0, p - window + 1), p].
//
// One warp a (new token, query head): 32 keys at a time, a lane a key for the
// scores and a slice of head_dim for the sum over them.
#include <cmath>

#include "pa_fp4.cuh"
#include "pa_host.h"

namespace pa {

namespace {

struct Args {
  const uint16_t* q;
  uint16_t* out;
  const uint8_t* kc;
  const uint8_t* vc;
  const int32_t* bt;
  const int32_t* seq_lens;
  const int32_t* query_start;
  int32_t* err;
  long long num_blocks, total_q;
  int num_seqs, stride, Hq, H, G, log2B, window;
  float scale, v_scale;
};

constexpr int kWarps = 4;

// 16 consecutive elements of a row, in fp32
template <int D, bool kFour>
__device__ __forceinline__ void load16(const Args& a, const uint8_t* pool, int block, int h, int r,
                                       int g, float (&x)[16]) {
  const int B = 1 << a.log2B;
  if constexpr (kFour) {
    const uint8_t* plane = pool + fp4_plane(block, a.H, h, B * fp4_row_bytes(D));
    const uint2 w = *reinterpret_cast<const uint2*>(plane + r * (D / 2) + 8 * g);
    const uint32_t s8 = plane[fp4_scale_off<D>(B, r, g)];
    const float s = unpack2<false>(e4m3x2_to_f16x2(s8)).x;
    uint32_t f[8];
    e2m1x8_to_f16x2(w.x, *reinterpret_cast<uint32_t(*)[4]>(f));
    e2m1x8_to_f16x2(w.y, *reinterpret_cast<uint32_t(*)[4]>(f + 4));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 y = unpack2<false>(f[i]);
      x[2 * i] = y.x * s;
      x[2 * i + 1] = y.y * s;
    }
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(
        pool + (((size_t)block * B + r) * a.H + h) * D + 16 * g);
    const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo, hi;
      e4m3x4_to_f16x2x2(c[i], lo, hi);
      const float2 u = unpack2<false>(lo), v = unpack2<false>(hi);
      x[4 * i] = u.x; x[4 * i + 1] = u.y; x[4 * i + 2] = v.x; x[4 * i + 3] = v.y;
    }
  }
}

template <int D, bool kBF16, bool kFour>
__global__ void __launch_bounds__(32 * kWarps) prefill_quant_kernel(const Args a) {
  __shared__ float qs[kWarps][D];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long unit = (long long)blockIdx.x * kWarps + warp;
  const long long row = unit / a.Hq;
  const int hq = (int)(unit % a.Hq), h = hq / a.G;
  if (row >= a.total_q) return;
  // the sequence: the last one that starts at or before the row
  int lo = -1, hi = a.num_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((long long)__ldg(a.query_start + mid) <= row) lo = mid;
    else hi = mid;
  }
  if (lo < 0) return;
  const long long q0 = __ldg(a.query_start + lo), q1 = __ldg(a.query_start + lo + 1);
  if (row >= q1) return;
  const int T = __ldg(a.seq_lens + lo);
  uint16_t* const out = a.out + ((size_t)row * a.Hq + hq) * D;
  if (q0 < 0 || q1 > a.total_q || T < 0 || (long long)T > ((long long)a.stride << a.log2B) ||
      q1 - q0 > T) {
    if (lane == 0) set_error(a.err, PA_DEVERR_SEQ_LEN);
    for (int d = lane; d < D; d += 32) out[d] = 0;
    return;
  }
  const int p = (int)(T - (q1 - q0) + (row - q0));
  const int first = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
  for (int d = lane; d < D / 2; d += 32) {
    const float2 y = unpack2<kBF16>(
        reinterpret_cast<const uint32_t*>(a.q + ((size_t)row * a.Hq + hq) * D)[d]);
    qs[warp][2 * d] = y.x;
    qs[warp][2 * d + 1] = y.y;
  }
  __syncwarp();
  constexpr int V = D / 32;   // output elements a lane: d = V lane ..
  float m = -INFINITY, l = 0.f, o[V] = {};
  bool nan = false;
  for (int t0 = first & ~31; t0 <= p; t0 += 32) {
    const int t = t0 + lane;
    float s = -INFINITY;
    int block = -1;
    if (t >= first && t <= p) {
      block = __ldg(a.bt + (size_t)lo * a.stride + (t >> a.log2B));
      if (block < 0 || (long long)block >= a.num_blocks) {
        set_error(a.err, PA_DEVERR_BLOCK_ID);
        block = -1;
      }
    }
    const int r = t & ((1 << a.log2B) - 1);
    if (block >= 0) {
      s = 0.f;
      for (int g = 0; g < D / 16; ++g) {
        float x[16];
        load16<D, kFour>(a, a.kc, block, h, r, g, x);
        for (int i = 0; i < 16; ++i) s = fmaf(x[i], qs[warp][16 * g + i], s);
      }
      s *= a.scale;
    }
    float mx = s;
    for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    const float mn = fmaxf(m, mx);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float alpha = expf(m - base), w = expf(s - base);
    m = mn;
    l = l * alpha + w;
    for (int e = 0; e < V; ++e) o[e] *= alpha;
    for (int k = 0; k < 32; ++k) {
      const int b = __shfl_sync(0xffffffffu, block, k);
      const float wk = __shfl_sync(0xffffffffu, w, k);
      if (b < 0) continue;
      float x[16];
      load16<D, kFour>(a, a.vc, b, h, (t0 + k) & ((1 << a.log2B) - 1), V * lane / 16, x);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        nan |= x[i] != x[i];
        if (i / V == lane % (16 / V)) o[i % V] = fmaf(wk, x[i], o[i % V]);
      }
    }
  }
  for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  nan = __any_sync(0xffffffffu, nan) != 0;
  const float mul = nan ? __uint_as_float(0x7fffffffu) : (l == 0.f ? 0.f : a.v_scale / l);
  for (int e = 0; e < V; ++e) out[V * lane + e] = round16<kBF16>(o[e] * mul);
}

int check_shape(int Hq, int H, int D) {
  if (Hq <= 0 || H <= 0 || Hq % H != 0) return PA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return PA_ERR_UNSUPPORTED;
  if (Hq / H > 16) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

template <bool kFour>
int prefill_quant(const void* q, const void* k_cache, const void* v_cache,
                  const int32_t* block_tables, int32_t table_stride, const int32_t* seq_lens,
                  const int32_t* query_start, int32_t num_seqs, int64_t total_q,
                  int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                  int64_t num_blocks, int32_t q_dtype, float scale, float k_scale, float v_scale,
                  int32_t window, void* out, void* workspace, size_t workspace_bytes,
                  int32_t* err_word, pa_stream stream) {
  if (num_seqs < 0 || total_q < 0 || table_stride < 0 || num_blocks < 0 || window < 0)
    return PA_ERR_INVALID_ARG;
  if (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) ||
      !std::isfinite(v_scale) || !std::isfinite(scale))
    return PA_ERR_INVALID_ARG;
  if (q_dtype != PA_F16 && q_dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (!is_pow2(block_size) || block_size < 4 || block_size > 256) return PA_ERR_UNSUPPORTED;
  size_t need = 0;
  if (int rc = pa_prefill_quant_workspace_size(num_q_heads, num_kv_heads, head_dim, &need))
    return rc;
  // a block's bytes are counted in 31 bits
  if ((long long)num_kv_heads * block_size * head_dim > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_q == 0) return PA_OK;
  if (total_q > 0x7fffffffLL || num_blocks > 0x7fffffffLL) return PA_ERR_INVALID_ARG;
  if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !query_start || !out ||
      !workspace || out == q)
    return PA_ERR_INVALID_ARG;
  if (num_blocks == 0 || table_stride == 0) return PA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned16(workspace))
    return PA_ERR_INVALID_ARG;
  if (workspace_bytes < need) return PA_ERR_WORKSPACE;
  Args a{};
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.kc = static_cast<const uint8_t*>(k_cache);
  a.vc = static_cast<const uint8_t*>(v_cache);
  a.bt = block_tables;
  a.seq_lens = seq_lens;
  a.query_start = query_start;
  a.err = err_word;
  a.num_blocks = num_blocks;
  a.total_q = total_q;
  a.num_seqs = num_seqs;
  a.stride = table_stride;
  a.Hq = num_q_heads;
  a.H = num_kv_heads;
  a.G = num_q_heads / num_kv_heads;
  a.log2B = ilog2(block_size);
  a.window = window;
  a.scale = scale * k_scale;
  a.v_scale = v_scale;
  const long long units = (long long)total_q * num_q_heads;
  const dim3 grid((unsigned)((units + kWarps - 1) / kWarps)), block(32 * kWarps);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = q_dtype == PA_BF16;
  clear_stale_error();
  cudaError_t e;
  if (head_dim == 64)
    e = bf16 ? launch_pdl(prefill_quant_kernel<64, true, kFour>, grid, block, 0, s, a)
             : launch_pdl(prefill_quant_kernel<64, false, kFour>, grid, block, 0, s, a);
  else
    e = bf16 ? launch_pdl(prefill_quant_kernel<128, true, kFour>, grid, block, 0, s, a)
             : launch_pdl(prefill_quant_kernel<128, false, kFour>, grid, block, 0, s, a);
  return launch_status(e, "quantized prefill launch");
}

}  // namespace

}  // namespace pa

using namespace pa;

extern "C" {

int pa_prefill_quant_workspace_size(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                    size_t* bytes) {
  if (!bytes) return PA_ERR_INVALID_ARG;
  if (int rc = check_shape(num_q_heads, num_kv_heads, head_dim)) return rc;
  *bytes = PA_PREFILL_QUANT_COUNTERS;
  return PA_OK;
}

int pa_prefill_fp8(const void* q, const void* k_cache, const void* v_cache,
                   const int32_t* block_tables, int32_t table_stride, const int32_t* seq_lens,
                   const int32_t* query_start, int32_t num_seqs, int64_t total_q,
                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                   int32_t block_size, int64_t num_blocks, int32_t q_dtype, float scale,
                   float k_scale, float v_scale, int32_t window, void* out, void* workspace,
                   size_t workspace_bytes, int32_t* err_word, pa_stream stream) {
  return prefill_quant<false>(q, k_cache, v_cache, block_tables, table_stride, seq_lens,
                              query_start, num_seqs, total_q, num_q_heads, num_kv_heads, head_dim,
                              block_size, num_blocks, q_dtype, scale, k_scale, v_scale, window,
                              out, workspace, workspace_bytes, err_word, stream);
}

int pa_prefill_fp4(const void* q, const void* k_cache, const void* v_cache,
                   const int32_t* block_tables, int32_t table_stride, const int32_t* seq_lens,
                   const int32_t* query_start, int32_t num_seqs, int64_t total_q,
                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                   int32_t block_size, int64_t num_blocks, int32_t q_dtype, float scale,
                   float k_scale, float v_scale, int32_t window, void* out, void* workspace,
                   size_t workspace_bytes, int32_t* err_word, pa_stream stream) {
  return prefill_quant<true>(q, k_cache, v_cache, block_tables, table_stride, seq_lens,
                             query_start, num_seqs, total_q, num_q_heads, num_kv_heads, head_dim,
                             block_size, num_blocks, q_dtype, scale, k_scale, v_scale, window,
                             out, workspace, workspace_bytes, err_word, stream);
}

}  // extern "C"
