// From the projection to the cache: norms of query and key heads, the position
// rotation, and the store of keys and values at their slots; the 4-bit cache's
// write and read-back.
//
// Formulas (fp32 throughout, each operation rounded once; x is the 16-bit input):
//   norm      y_d = x_d * r * w_d,  r = 1 / sqrt(mean_d(x_d^2) + eps)
//   rotation  a' = a c - b s,  b' = b c + a s  for the pairs (a, b) =
//             (y_i, y_{i + rot/2}), or (y_{2i}, y_{2i+1}) when interleaved,
//             i < rot / 2, with c, s the position's row of the angle table
//   store     round to 16 bits; an E4M3 or E2M1 pool quantizes that 16-bit value
// The products of the rotation are rounded before they are added (no fused
// multiply-add), so that the result is the same on every path that writes it.
//
// Bound: bytes.  A token of 32 query and 8 KV heads of 128 moves 24.6 KB
// between q, k, v, the pools and the rotated queries, and computes 3 operations
// an element.  A row (one head of one token) is held by D / 8 lanes of 16 bytes
// each, so loads and stores are whole 16-byte vectors and the rotation's partner
// element is in the lane rot / 16 away (four shuffles a row); the angles are
// loaded once per thread and used for all of the token's rows.
#include <cmath>

#include "pa_fp4.cuh"
#include "pa_host.h"

namespace pa {

namespace {

enum Pool : int { kPool16 = 0, kPoolE4M3 = 1, kPoolE2M1 = 2 };

struct AppendArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  long long q_stride, k_stride, v_stride;   // elements between tokens
  const float* cos_sin;                     // [max_pos][rot]: rot / 2 cosines, then sines
  int rot, max_pos, interleaved;
  const uint16_t* q_norm;
  const uint16_t* k_norm;
  float eps;
  const int32_t* bt;
  int stride, num_seqs;
  const int32_t* tok_seq;
  const int32_t* tok_pos;
  const int64_t* slots_in;                  // given slots instead of tables (write only)
  uint16_t* q_out;
  uint8_t* kc;
  uint8_t* vc;
  long long num_blocks;
  int log2B, Hq, H;
  float k_scale, v_scale;
  int64_t* slots;
  int32_t* err;
};

constexpr int kThreads = 256;

// The slot of token `tok`, or -1 for a token that writes nothing: a padding
// token (sequence -1, or a negative given slot), or a bad one, which sets an
// error bit (thread 0 reports).  pos receives its position.
__device__ __forceinline__ long long append_slot(const AppendArgs& a, long long tok, int& pos) {
  const bool report = threadIdx.x == 0 && blockIdx.y == 0;
  if (a.slots_in) {
    const long long s = a.slots_in[tok];
    pos = 0;
    if (s >= (a.num_blocks << a.log2B)) {
      if (report) set_error(a.err, PA_DEVERR_SLOT);
      return -1;
    }
    return s < 0 ? -1 : s;
  }
  const int i = a.tok_seq[tok];
  pos = a.tok_pos[tok];
  if (i == -1) return -1;
  if (i < 0 || i >= a.num_seqs || pos < 0 || (long long)pos >= ((long long)a.stride << a.log2B) ||
      (a.rot > 0 && pos >= a.max_pos)) {
    if (report) set_error(a.err, PA_DEVERR_POSITION);
    return -1;
  }
  const int p = a.bt[(size_t)i * a.stride + (pos >> a.log2B)];
  if (p < 0 || (long long)p >= a.num_blocks) {
    if (report) set_error(a.err, PA_DEVERR_BLOCK_ID);
    return -1;
  }
  return ((long long)p << a.log2B) + (pos & ((1 << a.log2B) - 1));
}

// One block per token (blockIdx.x) and share of its rows (blockIdx.y).  Rows
// are the Hq query heads, then the H key heads, then the H value heads.
template <int D, bool kBF16, int kPool, bool kNorm>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a) {
  constexpr int LPR = D / 8;               // lanes per row
  constexpr int RPP = kThreads / LPR;      // rows per pass of the block
  grid_dep_wait();
  grid_dep_launch();
  const long long tok = blockIdx.x;
  const int j = threadIdx.x % LPR;         // this lane's head_dim 8 j .. 8 j + 7
  const int d0 = 8 * j;
  const int rows = a.Hq + 2 * a.H;
  int pos;
  const long long slot = append_slot(a, tok, pos);
  if (a.slots && threadIdx.x == 0 && blockIdx.y == 0) a.slots[tok] = slot;
  if (slot < 0) return;                    // the whole block: every thread found the same slot

  // this lane's angles, the sine with the sign of its own product
  const int half = a.rot >> 1;
  const bool turns = d0 < a.rot;
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) c[e] = s[e] = 0.f;
  if (turns) {
    const float* cs = a.cos_sin + (size_t)pos * a.rot;
    if (a.interleaved) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs + d0 / 2));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(cs + half + d0 / 2));
      c[0] = c[1] = c4.x; c[2] = c[3] = c4.y; c[4] = c[5] = c4.z; c[6] = c[7] = c4.w;
      s[0] = -s4.x; s[1] = s4.x; s[2] = -s4.y; s[3] = s4.y;
      s[4] = -s4.z; s[5] = s4.z; s[6] = -s4.w; s[7] = s4.w;
    } else {
      const bool first = d0 < half;
      const int i0 = first ? d0 : d0 - half;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs + i0 + 4 * u));
        const float4 s4 = __ldg(reinterpret_cast<const float4*>(cs + half + i0 + 4 * u));
        c[4 * u] = c4.x; c[4 * u + 1] = c4.y; c[4 * u + 2] = c4.z; c[4 * u + 3] = c4.w;
        s[4 * u] = first ? -s4.x : s4.x;
        s[4 * u + 1] = first ? -s4.y : s4.y;
        s[4 * u + 2] = first ? -s4.z : s4.z;
        s[4 * u + 3] = first ? -s4.w : s4.w;
      }
    }
  }
  // the lane that holds the partner elements (this one when interleaved)
  const int lane = threadIdx.x & 31;
  int partner = lane;
  if (turns && !a.interleaved) partner = d0 < half ? lane + half / 8 : lane - half / 8;

  const int r0 = blockIdx.y * RPP + threadIdx.x / LPR, step = gridDim.y * RPP;
  // rows in lockstep over the warp (the shuffles need every lane)
  const int passes = (rows - (int)(blockIdx.y * RPP) + step - 1) / step;
  for (int it = 0; it < passes; ++it) {
    const int r = r0 + it * step;
    const bool in = r < rows;
    const int h = r < a.Hq ? r : (r < a.Hq + a.H ? r - a.Hq : r - a.Hq - a.H);
    const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.H;
    uint4 x4 = make_uint4(0u, 0u, 0u, 0u);
    if (in) {
      const uint16_t* src = is_q ? a.q + tok * a.q_stride
                                 : (is_v ? a.v + tok * a.v_stride : a.k + tok * a.k_stride);
      x4 = *reinterpret_cast<const uint4*>(src + h * D + d0);
    }
    const uint32_t w[4] = {x4.x, x4.y, x4.z, x4.w};
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<kBF16>(w[i]);
      y[2 * i] = f.x;
      y[2 * i + 1] = f.y;
    }
    if constexpr (kNorm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const uint16_t* nw = is_q ? a.q_norm : a.k_norm;
      if (in && !is_v && nw) {
        const float inv = __frsqrt_rn(ss * (1.f / D) + a.eps);
        const uint4 g4 = __ldg(reinterpret_cast<const uint4*>(nw + d0));
        const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 g = unpack2<kBF16>(gw[i]);
          y[2 * i] = y[2 * i] * inv * g.x;
          y[2 * i + 1] = y[2 * i + 1] * inv * g.y;
        }
      }
    }
    if (a.rot > 0) {
      float p[8];
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = y[e ^ 1];
      } else if constexpr (kNorm) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = __shfl_sync(0xffffffffu, y[e], partner);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack2<kBF16>(__shfl_sync(0xffffffffu, w[i], partner));
          p[2 * i] = f.x;
          p[2 * i + 1] = f.y;
        }
      }
      if (turns && !is_v) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          y[e] = __fadd_rn(__fmul_rn(y[e], c[e]), __fmul_rn(p[e], s[e]));
      }
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack2<kBF16>(y[2 * i], y[2 * i + 1]);
    if (in && is_q)
      *reinterpret_cast<uint4*>(a.q_out + ((size_t)tok * a.Hq + h) * D + d0) =
          make_uint4(o[0], o[1], o[2], o[3]);
    if constexpr (kPool == kPool16) {
      if (in && !is_q)
        *reinterpret_cast<uint4*>((is_v ? a.vc : a.kc) + (((size_t)slot * a.H + h) * D + d0) * 2) =
            make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      const float scale = is_v ? a.v_scale : a.k_scale;
      float z[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<kBF16>(o[i]);
        z[2 * i] = f.x;
        z[2 * i + 1] = f.y;
      }
      if constexpr (kPool == kPoolE4M3) {
        uint32_t e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          e[i] = f32x2_to_e4m3x2(__fdiv_rn(z[2 * i], scale), __fdiv_rn(z[2 * i + 1], scale));
        if (in && !is_q)
          *reinterpret_cast<uint2*>((is_v ? a.vc : a.kc) + ((size_t)slot * a.H + h) * D + d0) =
              make_uint2(e[0] | (e[1] << 16), e[2] | (e[3] << 16));
      } else {
        // the group of 16 is this lane's 8 values and its neighbour's
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(z[e]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const uint32_t s8 = f32x2_to_e4m3x2(__fdiv_rn(m, __fmul_rn(6.f, scale)), 0.f) & 0xffu;
        const float d = __fmul_rn(unpack2<false>(e4m3x2_to_f16x2(s8)).x, scale);
        uint32_t code = 0u;
        if (d > 0.f) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            code |= f32x2_to_e2m1x2(__fdiv_rn(z[2 * i], d), __fdiv_rn(z[2 * i + 1], d)) << (8 * i);
        }
        if (in && !is_q) {
          const int B = 1 << a.log2B, row = (int)(slot & (B - 1));
          uint8_t* plane =
              (is_v ? a.vc : a.kc) + fp4_plane(slot >> a.log2B, a.H, h, B * fp4_row_bytes(D));
          *reinterpret_cast<uint32_t*>(plane + row * (D / 2) + 4 * j) = code;
          if ((j & 1) == 0) plane[fp4_scale_off<D>(B, row, j >> 1)] = (uint8_t)s8;
        }
      }
    }
  }
}

struct ReadArgs {
  const int64_t* slots;
  const uint8_t* kc;
  const uint8_t* vc;
  uint16_t* k_out;
  uint16_t* v_out;
  long long n, num_blocks;
  int log2B, H;
  float k_scale, v_scale;
  int32_t* err;
};

// Rows at given slots of 4-bit pools as 16-bit values, code * scale16 (exact in
// fp32) * tensor scale, rounded to fp32 and then to 16 bits.  One block per
// token, D / 8 lanes per row as in the write.
template <int D, bool kBF16>
__global__ void __launch_bounds__(kThreads) read_fp4_kernel(const ReadArgs a) {
  constexpr int LPR = D / 8;
  grid_dep_wait();
  grid_dep_launch();
  const long long tok = blockIdx.x;
  const long long s = a.slots[tok];
  if (s < 0) return;
  if (s >= (a.num_blocks << a.log2B)) {
    if (threadIdx.x == 0) set_error(a.err, PA_DEVERR_SLOT);
    return;
  }
  const int B = 1 << a.log2B, row = (int)(s & (B - 1));
  const int j = threadIdx.x % LPR;
  for (int r = threadIdx.x / LPR; r < 2 * a.H; r += kThreads / LPR) {
    const bool is_v = r >= a.H;
    const int h = is_v ? r - a.H : r;
    const uint8_t* plane =
        (is_v ? a.vc : a.kc) + fp4_plane(s >> a.log2B, a.H, h, B * fp4_row_bytes(D));
    const uint32_t code = *reinterpret_cast<const uint32_t*>(plane + row * (D / 2) + 4 * j);
    const uint32_t s8 = plane[fp4_scale_off<D>(B, row, j >> 1)];
    const float s16 = unpack2<false>(e4m3x2_to_f16x2(s8)).x;
    const float scale = is_v ? a.v_scale : a.k_scale;
    uint32_t f[4], o[4];
    e2m1x8_to_f16x2(code, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 g = unpack2<false>(f[i]);
      o[i] = pack2<kBF16>(g.x * s16 * scale, g.y * s16 * scale);
    }
    *reinterpret_cast<uint4*>((is_v ? a.v_out : a.k_out) + ((size_t)tok * a.H + h) * D + 8 * j) =
        make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <int D, bool kBF16, int kPool>
cudaError_t launch_append_n(const AppendArgs& a, bool norm, dim3 grid, cudaStream_t s) {
  return norm ? launch_pdl(append_kernel<D, kBF16, kPool, true>, grid, dim3(kThreads), 0, s, a)
              : launch_pdl(append_kernel<D, kBF16, kPool, false>, grid, dim3(kThreads), 0, s, a);
}

template <int D, bool kBF16>
cudaError_t launch_append_p(const AppendArgs& a, int pool, bool norm, dim3 grid, cudaStream_t s) {
  if (pool == kPoolE2M1) return launch_append_n<D, kBF16, kPoolE2M1>(a, norm, grid, s);
  if (pool == kPoolE4M3) return launch_append_n<D, kBF16, kPoolE4M3>(a, norm, grid, s);
  return launch_append_n<D, kBF16, kPool16>(a, norm, grid, s);
}

int launch_append(const AppendArgs& a, int D, bool bf16, int pool, long long n, cudaStream_t s,
                  const char* what) {
  DeviceInfo di;
  if (int rc = current_device_info(&di)) return rc;
  // few tokens: a token's rows spread over several blocks, so that the step
  // takes one pass; many tokens fill the GPU by themselves
  const int per_pass = kThreads / (D / 8);
  const int passes = (a.Hq + 2 * a.H + per_pass - 1) / per_pass;
  long long y = n > 0 ? (2LL * di.sm_count + n - 1) / n : 1;
  if (y > passes) y = passes;
  if (y < 1) y = 1;
  const dim3 grid((unsigned)n, (unsigned)y);
  const bool norm = a.q_norm || a.k_norm;
  clear_stale_error();
  cudaError_t e;
  if (D == 64)
    e = bf16 ? launch_append_p<64, true>(a, pool, norm, grid, s)
             : launch_append_p<64, false>(a, pool, norm, grid, s);
  else
    e = bf16 ? launch_append_p<128, true>(a, pool, norm, grid, s)
             : launch_append_p<128, false>(a, pool, norm, grid, s);
  return launch_status(e, what);
}

bool scale_ok(float s) { return s > 0.f && std::isfinite(s) && std::isfinite(6.f * s); }

int append_shape(int32_t block_size, int32_t num_kv_heads, int32_t head_dim, int32_t src_dtype,
                 int32_t cache_dtype) {
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (num_kv_heads <= 0 || num_kv_heads > 65536) return PA_ERR_UNSUPPORTED;
  if (!is_pow2(block_size) || block_size > 256) return PA_ERR_UNSUPPORTED;
  if (src_dtype != PA_F16 && src_dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (cache_dtype != src_dtype && cache_dtype != PA_FP8_E4M3 && cache_dtype != PA_FP4_E2M1)
    return PA_ERR_UNSUPPORTED;
  if (cache_dtype == PA_FP4_E2M1 && block_size < 4) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

// The 4-bit write behind its two entry points: an append without queries,
// rotation or norms, of contiguous rows.
int write_fp4(const void* k, const void* v, int32_t src_dtype, AppendArgs a, int64_t num_tokens,
              void* k_cache, void* v_cache, int64_t num_blocks, int32_t block_size,
              int32_t num_kv_heads, int32_t head_dim, float k_scale, float v_scale,
              int32_t* err_word, pa_stream stream, const char* what) {
  if (num_tokens < 0 || num_blocks < 0) return PA_ERR_INVALID_ARG;
  if (int rc = append_shape(block_size, num_kv_heads, head_dim, src_dtype, PA_FP4_E2M1)) return rc;
  if (!scale_ok(k_scale) || !scale_ok(v_scale)) return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  if (num_tokens > 0x7fffffffLL) return PA_ERR_INVALID_ARG;
  if (!k || !v || !k_cache || !v_cache) return PA_ERR_INVALID_ARG;
  if (!a.slots_in && (!a.bt || !a.tok_seq || !a.tok_pos)) return PA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache))
    return PA_ERR_INVALID_ARG;
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_stride = a.v_stride = (long long)num_kv_heads * head_dim;
  a.kc = static_cast<uint8_t*>(k_cache);
  a.vc = static_cast<uint8_t*>(v_cache);
  a.num_blocks = num_blocks;
  a.log2B = ilog2(block_size);
  a.H = num_kv_heads;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.err = err_word;
  return launch_append(a, head_dim, src_dtype == PA_BF16, kPoolE2M1, num_tokens,
                       static_cast<cudaStream_t>(stream), what);
}

}  // namespace

}  // namespace pa

using namespace pa;

extern "C" {

int pa_append_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                   int64_t v_stride, int32_t src_dtype, const float* cos_sin, int32_t rotary_dim,
                   int32_t max_pos, int32_t interleaved, const void* q_norm, const void* k_norm,
                   float eps, const int32_t* block_tables, int32_t table_stride, int32_t num_seqs,
                   const int32_t* token_seq, const int32_t* token_pos, int64_t num_tokens,
                   void* q_out, void* k_cache, void* v_cache, int64_t num_blocks,
                   int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                   int32_t head_dim, int32_t cache_dtype, float k_scale, float v_scale,
                   int64_t* slot_mapping, int32_t* err_word, pa_stream stream) {
  if (num_tokens < 0 || num_seqs < 0 || table_stride < 0 || num_blocks < 0 || num_q_heads < 0 ||
      rotary_dim < 0 || max_pos < 0)
    return PA_ERR_INVALID_ARG;
  if (int rc = append_shape(block_size, num_kv_heads, head_dim, src_dtype, cache_dtype)) return rc;
  if (num_q_heads > 65536 || rotary_dim > head_dim || rotary_dim % 16 != 0)
    return PA_ERR_UNSUPPORTED;
  if ((q_norm || k_norm) && !(eps >= 0.f && std::isfinite(eps))) return PA_ERR_INVALID_ARG;
  if (cache_dtype != src_dtype && (!scale_ok(k_scale) || !scale_ok(v_scale)))
    return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  if (num_tokens > 0x7fffffffLL) return PA_ERR_INVALID_ARG;
  if (!k || !v || !block_tables || !token_seq || !token_pos || !k_cache || !v_cache)
    return PA_ERR_INVALID_ARG;
  if (num_q_heads > 0 && (!q || !q_out)) return PA_ERR_INVALID_ARG;
  if (rotary_dim > 0 && !cos_sin) return PA_ERR_INVALID_ARG;
  const int64_t kv_row = (int64_t)num_kv_heads * head_dim;
  if (k_stride < kv_row || v_stride < kv_row || k_stride % 8 || v_stride % 8)
    return PA_ERR_INVALID_ARG;
  if (num_q_heads > 0 && (q_stride < (int64_t)num_q_heads * head_dim || q_stride % 8))
    return PA_ERR_INVALID_ARG;
  const void* const ptrs[] = {q, k, v, cos_sin, q_norm, k_norm, q_out, k_cache, v_cache};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return PA_ERR_INVALID_ARG;
  AppendArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.cos_sin = cos_sin;
  a.rot = rotary_dim;
  a.max_pos = max_pos;
  a.interleaved = interleaved ? 1 : 0;
  a.q_norm = static_cast<const uint16_t*>(q_norm);
  a.k_norm = static_cast<const uint16_t*>(k_norm);
  a.eps = eps;
  a.bt = block_tables;
  a.stride = table_stride;
  a.num_seqs = num_seqs;
  a.tok_seq = token_seq;
  a.tok_pos = token_pos;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.kc = static_cast<uint8_t*>(k_cache);
  a.vc = static_cast<uint8_t*>(v_cache);
  a.num_blocks = num_blocks;
  a.log2B = ilog2(block_size);
  a.Hq = num_q_heads;
  a.H = num_kv_heads;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.slots = slot_mapping;
  a.err = err_word;
  const int pool = cache_dtype == PA_FP4_E2M1 ? kPoolE2M1
                                              : (cache_dtype == PA_FP8_E4M3 ? kPoolE4M3 : kPool16);
  return launch_append(a, head_dim, src_dtype == PA_BF16, pool, num_tokens,
                       static_cast<cudaStream_t>(stream), "append launch");
}

int pa_cache_write_fp4(const void* k, const void* v, int32_t src_dtype,
                       const int64_t* slot_mapping, int64_t num_tokens, void* k_cache,
                       void* v_cache, int64_t num_blocks, int32_t block_size,
                       int32_t num_kv_heads, int32_t head_dim, float k_scale, float v_scale,
                       int32_t* err_word, pa_stream stream) {
  AppendArgs a{};
  a.slots_in = slot_mapping;
  return write_fp4(k, v, src_dtype, a, num_tokens, k_cache, v_cache, num_blocks, block_size,
                   num_kv_heads, head_dim, k_scale, v_scale, err_word, stream,
                   "4-bit cache write launch");
}

int pa_cache_write_fp4_mapped(const void* k, const void* v, int32_t src_dtype,
                              const int32_t* block_tables, int32_t table_stride, int32_t num_seqs,
                              const int32_t* token_seq, const int32_t* token_pos,
                              int64_t num_tokens, void* k_cache, void* v_cache, int64_t num_blocks,
                              int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                              float k_scale, float v_scale, int64_t* slot_mapping,
                              int32_t* err_word, pa_stream stream) {
  if (num_seqs < 0 || table_stride < 0) return PA_ERR_INVALID_ARG;
  AppendArgs a{};
  a.bt = block_tables;
  a.stride = table_stride;
  a.num_seqs = num_seqs;
  a.tok_seq = token_seq;
  a.tok_pos = token_pos;
  a.slots = slot_mapping;
  return write_fp4(k, v, src_dtype, a, num_tokens, k_cache, v_cache, num_blocks, block_size,
                   num_kv_heads, head_dim, k_scale, v_scale, err_word, stream,
                   "slot-mapped 4-bit cache write launch");
}

int pa_cache_read_fp4(const int64_t* slot_mapping, int64_t num_tokens, const void* k_cache,
                      const void* v_cache, int64_t num_blocks, int32_t block_size,
                      int32_t num_kv_heads, int32_t head_dim, float k_scale, float v_scale,
                      void* k_out, void* v_out, int32_t out_dtype, int32_t* err_word,
                      pa_stream stream) {
  if (num_tokens < 0 || num_blocks < 0) return PA_ERR_INVALID_ARG;
  if (int rc = append_shape(block_size, num_kv_heads, head_dim, out_dtype, PA_FP4_E2M1)) return rc;
  if (!scale_ok(k_scale) || !scale_ok(v_scale)) return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  if (num_tokens > 0x7fffffffLL) return PA_ERR_INVALID_ARG;
  if (!slot_mapping || !k_cache || !v_cache || !k_out || !v_out) return PA_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_out) || !aligned16(v_out))
    return PA_ERR_INVALID_ARG;
  ReadArgs a{};
  a.slots = slot_mapping;
  a.kc = static_cast<const uint8_t*>(k_cache);
  a.vc = static_cast<const uint8_t*>(v_cache);
  a.k_out = static_cast<uint16_t*>(k_out);
  a.v_out = static_cast<uint16_t*>(v_out);
  a.n = num_tokens;
  a.num_blocks = num_blocks;
  a.log2B = ilog2(block_size);
  a.H = num_kv_heads;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.err = err_word;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)num_tokens), block(kThreads);
  const bool bf16 = out_dtype == PA_BF16;
  clear_stale_error();
  cudaError_t e;
  if (head_dim == 64)
    e = bf16 ? launch_pdl(read_fp4_kernel<64, true>, grid, block, 0, s, a)
             : launch_pdl(read_fp4_kernel<64, false>, grid, block, 0, s, a);
  else
    e = bf16 ? launch_pdl(read_fp4_kernel<128, true>, grid, block, 0, s, a)
             : launch_pdl(read_fp4_kernel<128, false>, grid, block, 0, s, a);
  return launch_status(e, "4-bit cache read launch");
}

}  // extern "C"
