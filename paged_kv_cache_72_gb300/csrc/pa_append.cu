// From the projection to the cache: norms of query and key heads, the position
// rotation, and the store of keys and values at their slots; the 4-bit cache's
// write and read-back.
//
// Formulas (fp32 throughout, each operation rounded once; x is the 16-bit input):
//   norm      y_d = x_d * r * w_d,  r = 1 / sqrt(mean_d(x_d^2) + eps)
//   rotation  a' = a c - b s,  b' = b c + a s  for the pairs (a, b) =
//             (y_i, y_{i + rot/2}), or (y_{2i}, y_{2i+1}) when interleaved,
//             i < rot / 2, with c, s the position's row of the angle table; with
//             axes, frequency i's c, s from the row of its axis's position
//   store     round to 16 bits; an E4M3 or E2M1 pool quantizes that 16-bit value
// Without a norm the products of the rotation are rounded before they are added
// (no fused multiply-add): bit for bit what separate products and a sum give.
//
// Bound: bytes.  A token of 32 query and 8 KV heads of 128 moves 24.6 KB
// between q, k, v, the pools and the rotated queries, and computes 3 operations
// an element.  8,192 of them (204 MB, half read, half written), with norms: 37.0
// us, 5.5 TB/s (a copy kernel of that size takes 34).  Into an E4M3 pool, 1,939
// tokens of 32 and 32 heads (80 MB): 16.6 us.  A step of 256 tokens takes 3.9 us,
// one of four 2.1.  A norm costs 8,192 tokens' stores into quantized pools 3 to 4
// us (E4M3 36.9 for 34.0, 4-bit 40.5 for 36.6).  With positions of three axes the
// 8,192 tokens take 43 us for 37.0 (a token's angles come from several rows of the
// table, and a norm's form spills up to 200 bytes a thread to hold them), 46.7 into a
// 4-bit pool (40.6 with one position), 42.5 into an E4M3 pool (36.9); 1,358 of 32 and 32
// heads, whole heads rotated, axes in turn, into an E4M3 pool 16.8 (with inputs repeated
// 14.0, with one position 12.7), 32 into a 4-bit pool 6.2 with the read-back, four 3.4.
//
// A row (one head of one token) is held by D / 8 lanes of 16 bytes each, so
// loads and stores are whole 16-byte vectors and the rotation's partner element
// is in the lane rot / 16 away (four shuffles a row).
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
  const uint8_t* axis_of;                   // [rot / 2]: the axis of every frequency
  const int32_t* rot_pos;                   // [axes][tokens]: positions that select angles
  int axes;
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

constexpr int kMaxAxes = 4;
constexpr int kThreads = 128;   // of a block of every kernel here (64 measured no better)

// The slot of token `tok`, or -1 for a token that writes nothing: a padding
// token (sequence -1, or a negative given slot), or a bad one, which sets an
// error bit (when `report`).  pos receives its position.
// kAxes: the position selects no angles.
template <bool kAxes = false>
__device__ __forceinline__ long long append_slot(const AppendArgs& a, long long tok, bool report,
                                                 int& pos) {
  if (a.slots_in) {
    const long long s = __ldg(a.slots_in + tok);
    pos = 0;
    if (s >= (a.num_blocks << a.log2B)) {
      if (report) set_error(a.err, PA_DEVERR_SLOT);
      return -1;
    }
    return s < 0 ? -1 : s;
  }
  const int i = __ldg(a.tok_seq + tok);
  pos = __ldg(a.tok_pos + tok);
  if (i == -1) return -1;
  if (i < 0 || i >= a.num_seqs || pos < 0 ||
      (long long)pos >= ((long long)a.stride << a.log2B) ||
      (!kAxes && a.rot > 0 && pos >= a.max_pos)) {
    if (report) set_error(a.err, PA_DEVERR_POSITION);
    return -1;
  }
  const int p = __ldg(a.bt + (size_t)i * a.stride + (pos >> a.log2B));
  if (p < 0 || (long long)p >= a.num_blocks) {
    if (report) set_error(a.err, PA_DEVERR_BLOCK_ID);
    return -1;
  }
  return ((long long)p << a.log2B) + (pos & ((1 << a.log2B) - 1));
}

// Two fp32 values at a time, each rounded as alone.
struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// scalar: a packed product and a packed sum may be contracted to one fused
// operation, __fadd_rn never is
__device__ __forceinline__ F2 add2(F2 a, F2 b) { return {__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)}; }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
// -x / d rounded to nearest, from r = 1 / d rounded to nearest: one residual
// step on -x r gives the correctly rounded quotient (P. Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990) where
// nothing under- or overflows: d within 2^+-100 and |x| at most 2^27 d
// (plain_quotient); an x so small that its residual is lost is far below the
// smallest code.  The negative quotient, because a residual of zero is +0: added
// to x r it would turn a quotient of -0 into +0; here it is multiplied by -r.
__device__ __forceinline__ F2 minus_div_by(F2 x, float d, float r) {
  const F2 y = mul2(x, {-r, -r});
  return fma2(fma2(y, {d, d}, x), {-r, -r}, y);
}
__device__ __forceinline__ bool plain_quotient(float largest, float d) {
  return d > 0x1p-100f && d < 0x1p100f && largest <= 0x1p27f * d;
}
// x / d for the others, off the common path (0 for d = 0)
__device__ __noinline__ float div_any(float x, float d) { return d > 0.f ? __fdiv_rn(x, d) : 0.f; }

// -z / d, four pairs of magnitudes up to `largest`; r is 1 / d rounded to nearest
__device__ __forceinline__ void minus_quotients(const F2 (&z)[4], float largest, float d, float r,
                                                F2 (&y)[4]) {
  if (plain_quotient(largest, d)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = minus_div_by(z[i], d, r);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = {-div_any(z[i].x, d), -div_any(z[i].y, d)};
  }
}

template <bool kBF16>
__device__ __forceinline__ void widen(const uint4& x, F2 (&y)[4]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<kBF16>(w[i]);
    y[i].x = f.x;
    y[i].y = f.y;
  }
}
template <bool kBF16>
__device__ __forceinline__ uint4 narrow(const F2 (&y)[4]) {
  return make_uint4(pack2<kBF16>(y[0].x, y[0].y), pack2<kBF16>(y[1].x, y[1].y),
                    pack2<kBF16>(y[2].x, y[2].y), pack2<kBF16>(y[3].x, y[3].y));
}

// What a lane needs to turn a position's rows: its 8 elements' cosines, the
// sines with the sign of their products, and the lane that holds the partners.
struct Turn {
  F2 c[4], s[4];
  int from;        // partner lane
  bool on, swap;   // this lane's elements turn; partners are neighbours

  __device__ __forceinline__ void load(const AppendArgs& a, int pos, int d0) {
    const int half = a.rot >> 1, lane = threadIdx.x & 31;
    on = d0 < a.rot;
    swap = a.interleaved != 0;
    from = lane;
    if (!on) return;
    const float* cs = a.cos_sin + (size_t)pos * a.rot;
    if (swap) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs + d0 / 2));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(cs + half + d0 / 2));
      c[0] = {c4.x, c4.x}; c[1] = {c4.y, c4.y}; c[2] = {c4.z, c4.z}; c[3] = {c4.w, c4.w};
      s[0] = {-s4.x, s4.x}; s[1] = {-s4.y, s4.y}; s[2] = {-s4.z, s4.z}; s[3] = {-s4.w, s4.w};
      return;
    }
    const bool first = d0 < half;
    from = first ? lane + (half >> 3) : lane - (half >> 3);
    const int i0 = first ? d0 : d0 - half;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs + i0 + 4 * u));
      float4 s4 = __ldg(reinterpret_cast<const float4*>(cs + half + i0 + 4 * u));
      if (first) s4 = make_float4(-s4.x, -s4.y, -s4.z, -s4.w);
      c[2 * u] = {c4.x, c4.y};
      c[2 * u + 1] = {c4.z, c4.w};
      s[2 * u] = {s4.x, s4.y};
      s[2 * u + 1] = {s4.z, s4.w};
    }
  }

  // load with a position per axis, at[x] on axis x: runs of four frequencies of
  // one axis as above, others one by one (they come from L1 or L2 like the rows)
  __device__ __forceinline__ void load_axes(const AppendArgs& a, const int (&at)[kMaxAxes],
                                            int d0) {
    const int half = a.rot >> 1, lane = threadIdx.x & 31;
    on = d0 < a.rot;
    swap = a.interleaved != 0;
    from = lane;
    if (!on) return;
    const bool first = d0 < half;
    const int i0 = swap ? d0 / 2 : (first ? d0 : d0 - half);
    if (!swap) from = first ? lane + (half >> 3) : lane - (half >> 3);
    float4 c4[2], s4[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (u == 1 && swap) break;
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(a.axis_of + i0 + 4 * u));
      const float* cs[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t x = (w >> (8 * e)) & 3u;
        const int pos = x == 0 ? at[0] : (x == 1 ? at[1] : (x == 2 ? at[2] : at[3]));
        cs[e] = a.cos_sin + (size_t)pos * a.rot + i0 + 4 * u + e;
      }
      if (w == (w & 0xffu) * 0x01010101u) {
        c4[u] = __ldg(reinterpret_cast<const float4*>(cs[0]));
        s4[u] = __ldg(reinterpret_cast<const float4*>(cs[0] + half));
      } else {
        c4[u] = make_float4(__ldg(cs[0]), __ldg(cs[1]), __ldg(cs[2]), __ldg(cs[3]));
        s4[u] = make_float4(__ldg(cs[0] + half), __ldg(cs[1] + half), __ldg(cs[2] + half),
                            __ldg(cs[3] + half));
      }
    }
    if (swap) {
      c[0] = {c4[0].x, c4[0].x}; c[1] = {c4[0].y, c4[0].y};
      c[2] = {c4[0].z, c4[0].z}; c[3] = {c4[0].w, c4[0].w};
      s[0] = {-s4[0].x, s4[0].x}; s[1] = {-s4[0].y, s4[0].y};
      s[2] = {-s4[0].z, s4[0].z}; s[3] = {-s4[0].w, s4[0].w};
      return;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (first) s4[u] = make_float4(-s4[u].x, -s4[u].y, -s4[u].z, -s4[u].w);
      c[2 * u] = {c4[u].x, c4[u].y};
      c[2 * u + 1] = {c4[u].z, c4[u].w};
      s[2 * u] = {s4[u].x, s4[u].y};
      s[2 * u + 1] = {s4[u].z, s4[u].w};
    }
  }

  // the angles times a norm's weights: gc = g c, gs = g_partner s (c is g where
  // nothing turns); every lane takes part
  template <bool kBF16>
  __device__ __forceinline__ void join(const uint16_t* weights, bool rotates, int d0) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(weights + d0));
    F2 g[4], p[4];
    widen<kBF16>(w, g);
    if (rotates) partners<kBF16>(w, g, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = rotates && on ? mul2(g[i], c[i]) : g[i];
      if (rotates && on) s[i] = mul2(p[i], s[i]);
    }
  }

  // the partner elements of a row whose 16 bytes are x (every lane takes part)
  template <bool kBF16>
  __device__ __forceinline__ void partners(const uint4& x, const F2 (&y)[4], F2 (&p)[4]) const {
    if (swap) {
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = {y[i].y, y[i].x};
    } else {
      uint4 o;
      o.x = __shfl_sync(0xffffffffu, x.x, from);
      o.y = __shfl_sync(0xffffffffu, x.y, from);
      o.z = __shfl_sync(0xffffffffu, x.z, from);
      o.w = __shfl_sync(0xffffffffu, x.w, from);
      widen<kBF16>(o, p);
    }
  }
};

// One query or key row: norm (when `normed`), rotation, one rounding to 16
// bits.  Without a norm the products are rounded before they are added, as the
// header of this file says; with one t holds the angles times the weights
// (Turn::join) and the row is a' = r (x gc + p gs).
template <int D, bool kBF16, bool kNorm>
__device__ __forceinline__ uint4 turned(const AppendArgs& a, const uint4& x, const Turn& t,
                                        bool normed) {
  const bool rotates = a.rot > 0;
  F2 y[4], p[4];
  widen<kBF16>(x, y);
  if (rotates) t.partners<kBF16>(x, y, p);
  if (kNorm && normed) {
    F2 q = mul2(y[0], y[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) q = fma2(y[i], y[i], q);
    float ss = q.x + q.y;
#pragma unroll
    for (int k = 1; k < D / 8; k <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, k);
    const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = mul2(y[i], t.c[i]);
      if (rotates && t.on) y[i] = fma2(p[i], t.s[i], y[i]);
      y[i] = mul2(y[i], {r, r});
    }
  } else if (rotates && t.on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = add2(mul2(y[i], t.c[i]), mul2(p[i], t.s[i]));
  } else {
    return x;
  }
  return narrow<kBF16>(y);
}

// One key or value row into its pool, this lane's 16 bytes x of head h: as it
// is, as E4M3 codes, or as E2M1 codes whose group of 16 is this lane's 8 values
// and its neighbour's (every lane takes part).
template <int D, bool kBF16, int kPool>
__device__ __forceinline__ void store_row(uint8_t* pool, const uint4& x, long long slot, int H,
                                          int log2B, int h, float scale, bool in) {
  const int j = threadIdx.x % (D / 8), d0 = 8 * j;
  if constexpr (kPool == kPool16) {
    if (in) *reinterpret_cast<uint4*>(pool + (((size_t)slot * H + h) * D + d0) * 2) = x;
    return;
  }
  F2 z[4];
  widen<kBF16>(x, z);
  F2 y[4];
  float m = fmaxf(fabsf(z[0].x), fabsf(z[0].y));
#pragma unroll
  for (int i = 1; i < 4; ++i) m = max3f(m, fabsf(z[i].x), fabsf(z[i].y));
  // the scale's own reciprocals are the call's: the compiler hoists them; the
  // codes of the negative quotients get their sign bits flipped
  if constexpr (kPool == kPoolE4M3) {
    minus_quotients(z, m, scale, __frcp_rn(scale), y);
    uint32_t e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = f32x2_to_e4m3x2(y[i].x, y[i].y);
    if (in)
      *reinterpret_cast<uint2*>(pool + ((size_t)slot * H + h) * D + d0) =
          make_uint2((e[0] | (e[1] << 16)) ^ 0x80808080u, (e[2] | (e[3] << 16)) ^ 0x80808080u);
  } else if constexpr (kPool == kPoolE2M1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const float six = __fmul_rn(6.f, scale);
    const float s16 =
        plain_quotient(m, six) ? -minus_div_by({m, m}, six, __frcp_rn(six)).x : div_any(m, six);
    const uint32_t s8 = f32x2_to_e4m3x2(s16, 0.f) & 0xffu;
    const float d = __fmul_rn(unpack2<false>(e4m3x2_to_f16x2(s8)).x, scale);
    minus_quotients(z, m, d, __frcp_rn(d), y);
    const uint32_t code = 0x88888888u ^ f32x8_to_e2m1x8(y[0].x, y[0].y, y[1].x, y[1].y, y[2].x,
                                                        y[2].y, y[3].x, y[3].y);
    if (in) {
      const int B = 1 << log2B, row = (int)(slot & (B - 1));
      uint8_t* plane = pool + fp4_plane(slot >> log2B, H, h, B * fp4_row_bytes(D));
      *reinterpret_cast<uint32_t*>(plane + row * (D / 2) + 4 * j) = code;
      if ((j & 1) == 0) plane[fp4_scale_off<D>(B, row, j >> 1)] = (uint8_t)s8;
    }
  }
}

// Rows a thread group loads before it works on the first, and blocks of the
// append an SM (72 registers, a few of them spilled): 37.2 us for the append of
// 8,192 tokens; 3, 5 and 6 rows take 38.5, 38.8 and 43.8, five, six and eight
// blocks 40.6, 42.0 and 40.3.
constexpr int kBatch = 4;
constexpr int kBlocks = 7;

// Whether token `tok` can be rotated with axes: its positions, which `at` receives,
// lie in the table, and every frequency's axis is one of them (every lane of the
// warp takes part; a row's lanes read all of axis_of between them).
__device__ __forceinline__ bool axes_ok(const AppendArgs& a, long long tok, long long n, int d0,
                                        int (&at)[kMaxAxes]) {
  bool ok = true;
#pragma unroll
  for (int x = 0; x < kMaxAxes; ++x) {
    at[x] = x < a.axes ? __ldg(a.rot_pos + x * n + tok) : 0;
    ok = ok && at[x] >= 0 && (x >= a.axes || at[x] < a.max_pos);
  }
  if (2 * d0 < a.rot) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(a.axis_of + d0));
    const uint32_t most = (uint32_t)(a.axes - 1) * 0x01010101u;
    ok = ok && (__vcmpgtu4(w.x, most) | __vcmpgtu4(w.y, most)) == 0u;
  }
  return __all_sync(0xffffffffu, ok) != 0;
}

// One warp per token and share of its rows: query rows, then key rows with their
// value rows, each D / 8 lanes wide.  The angles are loaded once per lane and
// used for all of the share's rows; a norm's weights are multiplied into them, so
// that a normed row costs one multiplication more than a plain one.  The first
// rows of each kind are loaded before the token's slot is known.  A warp, not a
// block, per token: slot, angles and weights cost a warp some 400 instructions
// and three dependent loads, once for 24 passes of rows instead of four times
// (50 us with a block per token, 42 with a warp at the same six blocks an SM).
// kAxes: the angles of each frequency from the position on its axis.
template <int D, bool kBF16, int kPool, bool kNorm, bool kAxes>
__global__ void __launch_bounds__(kThreads, kBlocks)
    append_kernel(const AppendArgs a, int log2_shares, long long n) {
  constexpr int LPR = D / 8;               // lanes per row
  constexpr int RPP = 32 / LPR;            // rows per pass of a warp
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long unit = (long long)blockIdx.x * (kThreads / 32) + warp;
  const long long tok = unit >> log2_shares;
  const int shares = 1 << log2_shares, share = (int)unit & (shares - 1);
  if (tok >= n) return;
  const int d0 = 8 * (lane % LPR);
  const int r0 = share * RPP + lane / LPR, step = shares * RPP;
  const uint16_t* const qr = a.q + tok * a.q_stride + d0;
  const uint16_t* const kr = a.k + tok * a.k_stride + d0;
  const uint16_t* const vr = a.v + tok * a.v_stride + d0;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  uint4 xq[kBatch], xk = none, xv = none;
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int h = r0 + b * step;
    xq[b] = h < a.Hq ? *reinterpret_cast<const uint4*>(qr + h * D) : none;
  }
  if (r0 < a.H) {
    xk = *reinterpret_cast<const uint4*>(kr + r0 * D);
    xv = *reinterpret_cast<const uint4*>(vr + r0 * D);
  }
  int pos, at[kMaxAxes];
  const bool lead = lane == 0 && share == 0;
  long long slot = append_slot<kAxes>(a, tok, lead, pos);
  if constexpr (kAxes) {
    const bool ok = axes_ok(a, tok, n, d0, at);
    if (slot >= 0 && !ok) {
      if (lead) set_error(a.err, PA_DEVERR_POSITION);
      slot = -1;
    }
  }
  if (a.slots && lead) a.slots[tok] = slot;
  if (slot < 0) return;                    // the whole warp: every lane found the same slot
  Turn t;
  if constexpr (kAxes) t.load_axes(a, at, d0);
  else t.load(a, pos, d0);
  // rows in lockstep over the warp (the shuffles need every lane)
  if (kNorm && a.q_norm) t.join<kBF16>(a.q_norm, a.rot > 0, d0);
  uint16_t* const qo = a.q_out + (size_t)tok * a.Hq * D + d0;
  for (int first = share * RPP; first < a.Hq; first += kBatch * step) {
    const int hb = first + lane / LPR;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (first + b * step >= a.Hq) break;
      const int h = hb + b * step;
      const uint4 o = turned<D, kBF16, kNorm>(a, xq[b], t, a.q_norm != nullptr);
      if (h < a.Hq) *reinterpret_cast<uint4*>(qo + h * D) = o;
      const int next = h + kBatch * step;
      if (next < a.Hq) xq[b] = *reinterpret_cast<const uint4*>(qr + next * D);
    }
  }
  if constexpr (kNorm) {   // the keys' weights: the angles are read again (from L1)
    if (a.q_norm) {
      if constexpr (kAxes) t.load_axes(a, at, d0);
      else t.load(a, pos, d0);
    }
    if (a.k_norm) t.join<kBF16>(a.k_norm, a.rot > 0, d0);
  }
  for (int first = share * RPP; first < a.H; first += step) {
    const int h = first + lane / LPR;
    const bool in = h < a.H;
    const uint4 k = xk, v = xv;
    if (h + step < a.H) {
      xk = *reinterpret_cast<const uint4*>(kr + (h + step) * D);
      xv = *reinterpret_cast<const uint4*>(vr + (h + step) * D);
    }
    const uint4 o = turned<D, kBF16, kNorm>(a, k, t, a.k_norm != nullptr);
    store_row<D, kBF16, kPool>(a.kc, o, slot, a.H, a.log2B, h, a.k_scale, in);
    store_row<D, kBF16, kPool>(a.vc, v, slot, a.H, a.log2B, h, a.v_scale, in);
  }
}

// Rows of several tokens as one list, for kernels whose tokens have few rows:
// item i of a block's list is row i % rows of token i / rows, a thread group
// takes items RPP apart.
struct Items {
  int t, r, dt, dr, rows;
  __device__ __forceinline__ Items(int i, int stride, int rows_)
      : t(i / rows_), r(i % rows_), dt(stride / rows_), dr(stride % rows_), rows(rows_) {}
  __device__ __forceinline__ void next() {
    t += dt;
    r += dr;
    if (r >= rows) {
      r -= rows;
      ++t;
    }
  }
};

// The 4-bit write of rows that are rotated already, for tokens of few rows; bound
// by bytes (2 read and 0.5625 written for an element): H key rows, then H value
// rows of each of a block's per_block tokens.  All rows of a thread are in flight,
// at most kBatch of them (a token of few rows has no more, and tokens_per_block
// gives a block no more): their data and slots are loaded before the first is
// quantized.
template <int D, bool kBF16>
__global__ void __launch_bounds__(kThreads) write_fp4_kernel(const AppendArgs a, int per_block,
                                                             long long n) {
  constexpr int LPR = D / 8, RPP = kThreads / LPR;
  grid_dep_wait();
  grid_dep_launch();
  const int rows = 2 * a.H, j = threadIdx.x % LPR;
  const long long tok0 = (long long)blockIdx.x * per_block;
  const int tokens = (int)min((long long)per_block, n - tok0), count = tokens * rows;
  Items it(threadIdx.x / LPR, RPP, rows);
  uint4 x[kBatch];
  long long slot[kBatch];
  int h[kBatch];
  bool v[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const bool in = it.t < tokens;
    const long long tok = tok0 + it.t;
    v[b] = it.r >= a.H;
    h[b] = v[b] ? it.r - a.H : it.r;
    x[b] = make_uint4(0u, 0u, 0u, 0u);
    slot[b] = -1;
    if (in) {
      x[b] = *reinterpret_cast<const uint4*>((v[b] ? a.v : a.k) + tok * a.k_stride + h[b] * D +
                                             8 * j);
      const bool lead = j == 0 && it.r == 0;   // one thread a token
      int pos;
      slot[b] = append_slot(a, tok, lead, pos);
      if (a.slots && lead) a.slots[tok] = slot[b];
    }
    it.next();
  }
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    if (b * RPP >= count) break;
    store_row<D, kBF16, kPoolE2M1>(v[b] ? a.vc : a.kc, x[b], slot[b], a.H, a.log2B, h[b],
                                   v[b] ? a.v_scale : a.k_scale, slot[b] >= 0);
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
// binary16) * tensor scale, rounded to fp32 and then to 16 bits.  Bound by bytes
// and close behind them by issue slots (8,192 tokens of 8 heads of 128 out of memory,
// 43 MB: 9.9 us; 32,768: 30.2 us, 5.7 TB/s), so a lane takes 16 values of a row, 8 in
// each half (whole sectors a store): D / 16 lanes a row.  A block takes per_block
// tokens, kBatch rows a thread: their slots, then their codes, then their values.
template <int D, bool kBF16>
__global__ void __launch_bounds__(kThreads) read_fp4_kernel(const ReadArgs a, int per_block) {
  constexpr int LPR = D / 16, RPP = kThreads / LPR;
  grid_dep_wait();
  grid_dep_launch();
  const int B = 1 << a.log2B, rows = 2 * a.H, j = threadIdx.x % LPR;
  const long long tok0 = (long long)blockIdx.x * per_block;
  const int tokens = (int)min((long long)per_block, a.n - tok0), count = tokens * rows;
  Items it(threadIdx.x / LPR, RPP, rows);
  for (int i0 = 0; i0 < count; i0 += kBatch * RPP) {
    uint32_t code[kBatch][2], s8[kBatch][2];
    uint16_t* dst[kBatch];
    bool v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const long long tok = tok0 + it.t;
      v[b] = it.r >= a.H;
      const int h = v[b] ? it.r - a.H : it.r;
      dst[b] = nullptr;
      if (it.t < tokens) {
        const long long slot = __ldg(a.slots + tok);
        if (slot >= (a.num_blocks << a.log2B)) {
          if (j == 0 && it.r == 0) set_error(a.err, PA_DEVERR_SLOT);
        } else if (slot >= 0) {
          const uint8_t* plane = (v[b] ? a.vc : a.kc) +
                                 fp4_plane(slot >> a.log2B, a.H, h, B * fp4_row_bytes(D));
          const int row = (int)(slot & (B - 1));
          const uint8_t* codes = plane + row * (D / 2) + 4 * j;
          const uint8_t* scales = plane + fp4_scale_off<D>(B, row, j >> 1);
          code[b][0] = __ldg(reinterpret_cast<const uint32_t*>(codes));
          code[b][1] = __ldg(reinterpret_cast<const uint32_t*>(codes + D / 4));
          s8[b][0] = __ldg(scales);
          s8[b][1] = __ldg(scales + 4 * (D / 32));
          dst[b] = (v[b] ? a.v_out : a.k_out) + ((size_t)tok * a.H + h) * D + 8 * j;
        }
      }
      it.next();
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (!dst[b]) continue;
      const float scale = v[b] ? a.v_scale : a.k_scale;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t s16 = e4m3x2_to_f16x2(s8[b][half]);
        uint32_t f[4], o[4];
        e2m1x8_to_f16x2(code[b][half], f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 g = unpack2<false>(hmul2_lo(f[k], s16));
          const F2 y = mul2({g.x, g.y}, {scale, scale});
          o[k] = pack2<kBF16>(y.x, y.y);
        }
        *reinterpret_cast<uint4*>(dst[b] + half * (D / 2)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

// Tokens a block takes when a token has `rows` rows of `lanes`: as many as fill
// kBatch rows a thread, as long as two blocks an SM remain (write and read-back
// of 1,800 tokens of 2 heads of 64: 4.6 us, 6.4 with one token a block).
int tokens_per_block(int lanes, int rows, long long n, int sm_count) {
  long long t = (long long)kBatch * (kThreads / lanes) / rows;
  const long long most = n / (2LL * sm_count);
  if (t > most) t = most;
  return t < 1 ? 1 : (int)t;
}

template <int D, bool kBF16, int kPool, bool kNorm, bool kAxes>
cudaError_t launch_append_n(const AppendArgs& a, long long n, int sm_count, cudaStream_t s) {
  // shares of a token's rows, a power of two: until six warps an SM, and on to 32
  // warps an SM as long as a warp has more than 20 passes of rows (the 1,939 tokens
  // above: 16.8 us with two shares, 17.5 with four).  Up to 16: 4.6 us for 32
  // tokens of 64 and 8 heads into a 4-bit pool and back, 4.8 with 8, 5.5 with 4.
  // 32 and 8 heads of 128, norms, us with the rule's shares and with twice as many:
  // 256 tokens 4.0 (four) 4.0, 512 7.3 (two) 5.9, 1,024 12.2 (one) 9.3, 2,048 14.5
  // (one) 12.3, 4,096 20.2 (one) 21.8; 64 and 8 heads: 256 tokens 5.8 (four) 5.0,
  // 1,024 13.0 (two) 10.9, 2,048 17.6 (two) 19.3.  Between 512 and 2,048 tokens it
  // splits too little; a rule by passes and warps together is not built yet.
  const int per_pass = 32 / (D / 8), most = a.Hq > a.H ? a.Hq : a.H;
  const int passes = (a.Hq + a.H + per_pass - 1) / per_pass;
  int log2_shares = 0;
  while (log2_shares < 4 && (per_pass << log2_shares) < most) {
    const long long warps = n << log2_shares;
    if (warps >= 32LL * sm_count) break;
    if (warps >= 6LL * sm_count && (passes >> log2_shares) <= 20) break;
    ++log2_shares;
  }
  constexpr int kWarps = kThreads / 32;
  return launch_pdl(append_kernel<D, kBF16, kPool, kNorm, kAxes>,
                    dim3((unsigned)(((n << log2_shares) + kWarps - 1) / kWarps)), dim3(kThreads), 0, s,
                    a, log2_shares, n);
}

template <int D, bool kBF16, bool kAxes>
cudaError_t launch_append_p(const AppendArgs& a, int pool, long long n, int sm_count,
                            cudaStream_t s) {
  const bool norm = a.q_norm || a.k_norm;
  if (pool == kPoolE2M1)
    return norm ? launch_append_n<D, kBF16, kPoolE2M1, true, kAxes>(a, n, sm_count, s)
                : launch_append_n<D, kBF16, kPoolE2M1, false, kAxes>(a, n, sm_count, s);
  if (pool == kPoolE4M3)
    return norm ? launch_append_n<D, kBF16, kPoolE4M3, true, kAxes>(a, n, sm_count, s)
                : launch_append_n<D, kBF16, kPoolE4M3, false, kAxes>(a, n, sm_count, s);
  return norm ? launch_append_n<D, kBF16, kPool16, true, kAxes>(a, n, sm_count, s)
              : launch_append_n<D, kBF16, kPool16, false, kAxes>(a, n, sm_count, s);
}

template <bool kAxes>
int launch_append(const AppendArgs& a, int D, bool bf16, int pool, long long n, cudaStream_t s,
                  const char* what) {
  DeviceInfo di;
  if (int rc = current_device_info(&di)) return rc;
  clear_stale_error();
  cudaError_t e;
  if (D == 64)
    e = bf16 ? launch_append_p<64, true, kAxes>(a, pool, n, di.sm_count, s)
             : launch_append_p<64, false, kAxes>(a, pool, n, di.sm_count, s);
  else
    e = bf16 ? launch_append_p<128, true, kAxes>(a, pool, n, di.sm_count, s)
             : launch_append_p<128, false, kAxes>(a, pool, n, di.sm_count, s);
  return launch_status(e, what);
}

// a tensor scale; a 4-bit group's scale is a quotient by 6 s
bool scale_ok(float s, bool four_bit) {
  return s > 0.f && std::isfinite(s) && (!four_bit || std::isfinite(6.f * s));
}

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

// The 4-bit write behind its two entry points.
int write_fp4(const void* k, const void* v, int32_t src_dtype, AppendArgs a, int64_t num_tokens,
              void* k_cache, void* v_cache, int64_t num_blocks, int32_t block_size,
              int32_t num_kv_heads, int32_t head_dim, float k_scale, float v_scale,
              int32_t* err_word, pa_stream stream, const char* what) {
  if (num_tokens < 0 || num_blocks < 0) return PA_ERR_INVALID_ARG;
  if (int rc = append_shape(block_size, num_kv_heads, head_dim, src_dtype, PA_FP4_E2M1)) return rc;
  if (!scale_ok(k_scale, true) || !scale_ok(v_scale, true)) return PA_ERR_INVALID_ARG;
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
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // tokens of eight passes of a warp's rows or more: the append without queries
  // (4,096 tokens of 8 heads of 128: 8.9 us, 11.4 with the kernel below; 256
  // tokens 2.4 for 2.8, but 1,024 4.8 for 4.4); of fewer, several tokens to a block
  // (8,192 tokens of 2 heads of 64: 4.6 us, 7.8 with a warp or more a token; 256
  // tokens 2.0 for 3.0).  With two to seven passes a token, this is right up to
  // some 1,000 tokens (4 heads of 128, 256 tokens: 2.1 us for 2.2), the append
  // would be from there on (1,024: 3.1 for 3.7, 8,192: 10.0 for 11.5).
  constexpr int kFewLanes = 8 * 32;
  static_assert(kFewLanes <= kBatch * kThreads, "a token of few rows fits a block's registers");
  if (2 * num_kv_heads * (head_dim / 8) >= kFewLanes)
    return launch_append<false>(a, head_dim, src_dtype == PA_BF16, kPoolE2M1, num_tokens, s, what);
  DeviceInfo di;
  if (int rc = current_device_info(&di)) return rc;
  const int per = tokens_per_block(head_dim / 8, 2 * num_kv_heads, num_tokens, di.sm_count);
  const long long n = num_tokens;
  const dim3 grid((unsigned)((n + per - 1) / per)), block(kThreads);
  const bool bf16 = src_dtype == PA_BF16;
  clear_stale_error();
  cudaError_t e;
  if (head_dim == 64)
    e = bf16 ? launch_pdl(write_fp4_kernel<64, true>, grid, block, 0, s, a, per, n)
             : launch_pdl(write_fp4_kernel<64, false>, grid, block, 0, s, a, per, n);
  else
    e = bf16 ? launch_pdl(write_fp4_kernel<128, true>, grid, block, 0, s, a, per, n)
             : launch_pdl(write_fp4_kernel<128, false>, grid, block, 0, s, a, per, n);
  return launch_status(e, what);
}

// The append behind its two entry points; num_axes 0: one position a token.
int append(const uint8_t* axis_of, const int32_t* rot_pos, int32_t num_axes, const void* q,
           int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
           int32_t src_dtype, const float* cos_sin, int32_t rotary_dim, int32_t max_pos,
           int32_t interleaved, const void* q_norm, const void* k_norm, float eps,
           const int32_t* block_tables, int32_t table_stride, int32_t num_seqs,
           const int32_t* token_seq, const int32_t* token_pos, int64_t num_tokens, void* q_out,
           void* k_cache, void* v_cache, int64_t num_blocks, int32_t block_size,
           int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t cache_dtype,
           float k_scale, float v_scale, int64_t* slot_mapping, int32_t* err_word, pa_stream stream) {
  if (num_tokens < 0 || num_seqs < 0 || table_stride < 0 || num_blocks < 0 || num_q_heads < 0 ||
      rotary_dim < 0 || max_pos < 0)
    return PA_ERR_INVALID_ARG;
  if (int rc = append_shape(block_size, num_kv_heads, head_dim, src_dtype, cache_dtype)) return rc;
  if (num_q_heads > 65536 || rotary_dim > head_dim || rotary_dim % 16 != 0)
    return PA_ERR_UNSUPPORTED;
  if ((q_norm || k_norm) && !(eps >= 0.f && std::isfinite(eps))) return PA_ERR_INVALID_ARG;
  const bool four = cache_dtype == PA_FP4_E2M1;
  if (cache_dtype != src_dtype && (!scale_ok(k_scale, four) || !scale_ok(v_scale, four)))
    return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  if (num_tokens > 0x7fffffffLL) return PA_ERR_INVALID_ARG;
  if (!k || !v || !block_tables || !token_seq || !token_pos || !k_cache || !v_cache)
    return PA_ERR_INVALID_ARG;
  if (num_q_heads > 0 && (!q || !q_out)) return PA_ERR_INVALID_ARG;
  if (rotary_dim > 0 && !cos_sin) return PA_ERR_INVALID_ARG;
  if (num_axes && (!axis_of || !rot_pos || !aligned16(axis_of))) return PA_ERR_INVALID_ARG;
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
  a.axis_of = axis_of;
  a.rot_pos = rot_pos;
  a.axes = num_axes;
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
  const int pool = four ? kPoolE2M1 : (cache_dtype == PA_FP8_E4M3 ? kPoolE4M3 : kPool16);
  const bool bf16 = src_dtype == PA_BF16;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return num_axes ? launch_append<true>(a, head_dim, bf16, pool, num_tokens, s,
                                        "append (axes) launch")
                  : launch_append<false>(a, head_dim, bf16, pool, num_tokens, s, "append launch");
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
                   int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                   int32_t cache_dtype, float k_scale, float v_scale, int64_t* slot_mapping,
                   int32_t* err_word, pa_stream stream) {
  return append(nullptr, nullptr, 0, q, q_stride, k, k_stride, v, v_stride, src_dtype, cos_sin,
                rotary_dim, max_pos, interleaved, q_norm, k_norm, eps, block_tables, table_stride,
                num_seqs, token_seq, token_pos, num_tokens, q_out, k_cache, v_cache, num_blocks,
                block_size, num_q_heads, num_kv_heads, head_dim, cache_dtype, k_scale, v_scale,
                slot_mapping, err_word, stream);
}

int pa_append_rope_axes(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                        const void* v, int64_t v_stride, int32_t src_dtype, const float* cos_sin,
                        int32_t rotary_dim, int32_t max_pos, const uint8_t* axis_of,
                        const int32_t* rot_pos, int32_t num_axes, int32_t interleaved,
                        const void* q_norm, const void* k_norm, float eps,
                        const int32_t* block_tables, int32_t table_stride, int32_t num_seqs,
                        const int32_t* token_seq, const int32_t* token_pos, int64_t num_tokens,
                        void* q_out, void* k_cache, void* v_cache, int64_t num_blocks,
                        int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                        int32_t head_dim, int32_t cache_dtype, float k_scale, float v_scale,
                        int64_t* slot_mapping, int32_t* err_word, pa_stream stream) {
  if (num_axes < 1 || num_axes > kMaxAxes) return PA_ERR_UNSUPPORTED;
  if (rotary_dim <= 0) return PA_ERR_INVALID_ARG;
  return append(axis_of, rot_pos, num_axes, q, q_stride, k, k_stride, v, v_stride, src_dtype,
                cos_sin, rotary_dim, max_pos, interleaved, q_norm, k_norm, eps, block_tables,
                table_stride, num_seqs, token_seq, token_pos, num_tokens, q_out, k_cache, v_cache,
                num_blocks, block_size, num_q_heads, num_kv_heads, head_dim, cache_dtype, k_scale,
                v_scale, slot_mapping, err_word, stream);
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
  if (!scale_ok(k_scale, true) || !scale_ok(v_scale, true)) return PA_ERR_INVALID_ARG;
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
  DeviceInfo di;
  if (int rc = current_device_info(&di)) return rc;
  const int per = tokens_per_block(head_dim / 16, 2 * num_kv_heads, num_tokens, di.sm_count);
  const dim3 grid((unsigned)((num_tokens + per - 1) / per)), block(kThreads);
  const bool bf16 = out_dtype == PA_BF16;
  clear_stale_error();
  cudaError_t e;
  if (head_dim == 64)
    e = bf16 ? launch_pdl(read_fp4_kernel<64, true>, grid, block, 0, s, a, per)
             : launch_pdl(read_fp4_kernel<64, false>, grid, block, 0, s, a, per);
  else
    e = bf16 ? launch_pdl(read_fp4_kernel<128, true>, grid, block, 0, s, a, per)
             : launch_pdl(read_fp4_kernel<128, false>, grid, block, 0, s, a, per);
  return launch_status(e, "4-bit cache read launch");
}

}  // extern "C"
