// Paged single-query decode attention over a 4-bit (E2M1) KV cache.
//
// What it computes, with K and V the values the pool's codes stand for:
//   s_t = scale * k_scale * sum_d q_d codeK_td s16K_t(d/16)
//   o   = v_scale * sum_t softmax(s)_t codeV_t s16V_t(d/16),
// t over [max(0, T - window), T).  The tensor scales stay outside the products;
// code * s16 has at most 6 significant bits and lies in [2^-10, 2688], so it is
// exact in binary16, and every product is an f16 x f16 MMA with fp32 sums.
//
// Bound: bytes, and close behind them issue slots.  0.5625 bytes an element are
// read once and nothing else is, but a tile of 32 tokens also costs a warp 625
// instructions, 34 of them MMAs, 128 conversions and 128 multiplies by scales
// (head_dim 128, up to 4 heads a KV head; 5 to 8: 661, 52 of them MMAs).  32
// contexts of 16 to 32 K tokens, 8 KV heads of 128 (883 MB): 163 us with 32 query
// heads, 5.4 TB/s, 80% of a copy's rate, 181 us with 64; copies without arithmetic
// take 144 us.  256 contexts of 17 to 4,096 tokens, 32 over 8 heads (125 MB): 34.9
// us, of which 22 are tiles, 7 the start up to the first tile and 6 the joining of
// split contexts.  So:
//  * One warp is one pipeline.  A warp owns a (sequence, KV head) context or a
//    contiguous range of one.  Its tiles arrive in a ring of kStages tiles of
//    its own that it fills itself with 16-byte asynchronous copies, nine a lane
//    and tile: no producer, no barrier object, and no barrier between warps
//    until a block's end.  (One bulk copy a plane, with a barrier object a
//    stage, cost a warp 630 cycles a tile to issue against 480; loads straight
//    into fragments were slower than either.)
//  * Twelve warps, one block an SM.  Its warps get equal ranges and equal turns.
//    With three blocks of four warps the scheduler serves the oldest block
//    first, and the other two finish 7 and 15% later on a half-empty SM (11%
//    more time).
//  * Transposed products: S^T = K Q^T (16 tokens x 8 heads), O^T += V^T P^T
//    (16 head_dim rows x 8 heads), so that K and V are the A operands and 8
//    heads, not 16, fill a product; more than 8 heads a KV head take two tiles.
//  * The softmax's base is lazy (below), the weights' sums are one more MMA row
//    of ones, and tiles that need no mask run code without one (238 to 215 us
//    when they came in, together).
//
// Index maps (a contraction's order is free, an output row's place is undone
// at the write):
//  * a half tile is 16 tokens; MMA row r < 8 is token 4 (r / 2) + r % 2, row
//    8 + r the token two further.  The K rows of lane (gid, tig) = (lane / 4,
//    lane % 4) and its four V rows 4 tig .. 4 tig + 3 then each lie in one
//    group of four tokens: one scale word.
//  * S^T, k-step s: k index 2 tig + e stands for d = (D/4) tig + 4 s + e, and
//    2 tig + 8 + e for d + 2: the lane's K bytes are contiguous.
//  * O^T, m-tile i: row gid is d = (D/8) gid + 2 i, row gid + 8 the next: the
//    lane's V bytes are contiguous, and so is the slice of o it ends with.
//
// The split.  Every (sequence, KV head) is kStart units and one for each of its
// tiles; the units, in that order, are cut into equal contiguous ranges, one
// per block, and each block's range into one per warp.  A warp that holds a
// whole context writes it out.  The parts of contexts cut between the warps of
// a block are merged in shared memory; a context cut between blocks leaves one
// record (m, l, o) per block in the workspace, and the block that completes the
// context's count merges them, always in the order of the tiles.  No block
// waits for another.  Batches of short contexts take one warp each instead
// (kWhole).
//
// Roundings below fp32: the weights to a pair of binary16 values (2^-21), a
// bfloat16 query's elements under 2^-14 of its row's largest, and the output.
// Weights and the factors that join parts are ex2.approx (2^-22).
#include <cmath>
#include <mutex>

#include "pa_fp4.cuh"
#include "pa_host.h"

namespace pa {

namespace {

// Twelve warps leave a thread 168 registers, which o, the queries and a tile's
// work need; 16 warps of 128 spill and measured 1 to 2% more on long contexts and
// 2 to 8% on short ones (head_dim 64: 10%).  Two head tiles a KV head take 8 warps
// of 255 (12: 16 to 29% more).
__host__ __device__ constexpr int warps_of(int NH) { return NH == 1 ? 12 : 8; }
constexpr int kTile = 32;                 // tokens per tile
constexpr int kStages = 2;                // tiles in shared memory per warp (3: 0 to 4% more)
// Small batches take units / kLeast blocks, rounded up, so that each has about
// kLeast, one a scheduler: 8.4 us for one context of 300 tokens and one KV head, 8.9
// with 2 and with 8.
constexpr int kLeast = 4;
// A context's share of the work is its tiles and kStart for its start and end
// (queries to fragments, the write): without it a warp whose range holds many
// short contexts finishes last.  0 / 1 / 2 measured 86.2 / 60.9 / 61.8 us for
// 64 contexts of 1 to 2,048 tokens and 32 KV heads, 39.8 / 34.9 / 35.7 for the
// 256 contexts above.
constexpr int kStart = 1;
// Contexts of at most kWhole tiles go to one warp each when there are warps
// enough, which saves joining parts: 7.4 us for 8.6 with 16 contexts of 1 to 64
// tokens, 32 heads over 8, and 18.8 for 19.7 with 200 of 16 to 256 (12.5 for 10.5
// with 32 of 16 to 250, which leave most warps without one).
constexpr int kWhole = 8;
constexpr int kRecords = 4;               // of a split context, loaded at a time
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kUnitBits = 44, kCounted = 1 << 18;   // of the scanned sums; sequences it counts
// Weights are exp2(x - base) with base = a maximum less kShift, and a new base
// once they pass exp2(kShift + kLag) = 2^15, inside binary16's range.  A pair of
// binary16 values leaves 2^-25 of a small weight, whose second value is subnormal:
// the shift makes that 2^-33 of that maximum.  It cancels in o / l.
constexpr float kShift = 8.f, kLag = 7.f;

struct Args {
  const uint16_t* q;
  uint16_t* out;
  const uint8_t* kc;
  const uint8_t* vc;
  const int32_t* bt;
  const int32_t* seq_lens;
  uint32_t* ws_count;       // [PA_DECODE_MAX_CTAS], zero between calls
  float* ws_rec;            // [grid][2] records of rec_floats(G, D)
  int32_t* err;
  long long num_blocks;
  int num_seqs, stride, Hq, H, G, log2B, plane;
  float scale_log2, v_scale;
  int window, early_tables;
};

// o[G][D], m[G], l[G], padded to 16 bytes
__host__ __device__ constexpr size_t rec_floats(int G, int D) {
  return (size_t)G * D + (size_t)((2 * G + 3) & ~3);
}

__device__ __forceinline__ int clamp_len(int T, const Args& a) {
  return (T < 0 || (long long)T > ((long long)a.stride << a.log2B)) ? 0 : T;
}

__device__ __forceinline__ int first_token(int T, const Args& a) {
  return (a.window > 0 && T > a.window) ? T - a.window : 0;
}

// tiles of a context: from the tile that holds its first attended token
__device__ __forceinline__ int num_tiles(int T, const Args& a) {
  return (int)(((long long)T + kTile - 1) / kTile) - first_token(T, a) / kTile;
}

// kBytes from shared address addr + kOff
template <int kBytes, int kOff = 0>
__device__ __forceinline__ void ld_part(uint32_t addr, uint32_t* r) {
  if constexpr (kBytes == 16)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4 + %5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr), "n"(kOff));
  else if constexpr (kBytes == 8)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2 + %3];"
                 : "=r"(r[0]), "=r"(r[1])
                 : "r"(addr), "n"(kOff));
  else
    asm volatile("ld.shared.b32 %0, [%1 + %2];" : "=r"(r[0]) : "r"(addr), "n"(kOff));
}

// 16 bytes from global to shared memory, past L1; the lane's copies since the
// last commit are a group, and a wait leaves at most kPending groups in flight.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// a lane's part of the codes of kBs tokens of K and V (one tile's apart at dst)
template <int D, int kBs>
__device__ __forceinline__ void copy_codes(uint32_t dst, const uint8_t* k, const uint8_t* v) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    copy16(dst + 16 * kBs * i, k + 16 * kBs * i);
    copy16(dst + 16 * kBs * i + kTile * fp4_row_bytes(D), v + 16 * kBs * i);
  }
}
template <int kPending>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// A place in the list of tiles: tile k of head h of sequence i, and that
// sequence's length and tiles.
struct Walk {
  int i, h, k, T, nt;

  __device__ __forceinline__ void load_seq(const Args& a) {
    T = i < a.num_seqs ? clamp_len(__ldg(a.seq_lens + i), a) : 0;
    nt = num_tiles(T, a);
  }
  // the next tile; past the last sequence nt is 0
  __device__ __forceinline__ void advance(const Args& a) {
    if (++k < nt) return;
    k = 0;
    if (++h < a.H) return;
    h = 0;
    do {
      ++i;
      load_seq(a);
    } while (nt == 0 && i < a.num_seqs);
  }
};

// One warp's state over a range of one context's tiles.  The weights enter the
// products as a pair of binary16 values, their rounding and what it left: one
// value (2^-11) shows in outputs of either type (bfloat16 ones 8.5e-4 off a 32-bit
// computation's in norm, with the pair 3e-5 to 1.2e-4).  kTwin (at most 4 query
// heads): the 8 head columns hold the heads twice, the first copy's weights
// rounded, the second's the rest, so that the pair costs no second product; the
// two are added at the end.  With 32 contexts of 16 to 32 K tokens and 8 KV heads
// of 128, the pair takes 163 us for the 160 of one value with 4 query heads each,
// 181 for 161 with 8, and 137 for 118 with 16 heads to each of 4 KV heads.
template <int D, bool kBF16, int NH, bool kTwin>
struct Context {
  static constexpr int KS = D / 16;        // k-steps of S^T
  static constexpr int MT = D / 16;        // m-tiles of O^T
  static constexpr int KW = D / 32;        // words of K codes per lane and row
  static constexpr int VW = D / 64;        // words of V codes per lane and row
  static constexpr bool kPair = !kTwin;    // the pair takes two products
  uint32_t qb[NH][KS][2];
  float sl[NH][2];                         // score factor of heads 8 nh + 2 tig + e (log2)
  float o[NH][MT][4];
  float l[NH][4];                          // sums of the weights (rows alike)
  float base[NH][2];                       // weights are exp2(score - base)
  float limit;                             // weights above exp2(limit) move the base

  // The G query rows of this KV head as f16 fragments.  A bfloat16 row is
  // brought into binary16's range by a power of two (its largest magnitude
  // into [1, 2)), which the score factor takes back; elements 2^-14 below the
  // largest lose bits that are below 2^-24 of it.
  __device__ __forceinline__ void begin(const uint16_t* q, int G, float scale_log2) {
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      const int h = kTwin ? (gid & 3) : 8 * nh + gid;
      uint32_t w[D / 8];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (h < G) x = __ldg(reinterpret_cast<const uint4*>(q + (size_t)h * D + (D / 4) * tig) + c);
        w[4 * c] = x.x; w[4 * c + 1] = x.y; w[4 * c + 2] = x.z; w[4 * c + 3] = x.w;
      }
      float back = 1.f;
      if constexpr (kBF16) {
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const float2 f = unpack2<true>(w[i]);
          mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
        // 2^e <= mx < 2^(e+1); zero, subnormal or infinite maxima keep a
        // factor whose inverse is a normal number
        int e = (int)(__float_as_uint(mx) >> 23);
        e = min(max(e, 1), 253);
        back = __uint_as_float((uint32_t)e << 23);
        const float to = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const float2 f = unpack2<true>(w[i]);
          w[i] = pack2<false>(f.x * to, f.y * to);
        }
      }
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        qb[nh][s][0] = w[2 * s];
        qb[nh][s][1] = w[2 * s + 1];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sl[nh][e] = scale_log2 * __shfl_sync(kFull, back, 4 * (2 * tig + e));
        base[nh][e] = 0.f;
      }
      l[nh][0] = l[nh][1] = l[nh][2] = l[nh][3] = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i) o[nh][i][0] = o[nh][i][1] = o[nh][i][2] = o[nh][i][3] = 0.f;
    }
    limit = -INFINITY;
  }

  // scores of a tile: kc[hf] is the shared address of this lane's codes of half
  // hf (its first row; the second lies D bytes on), ks[hf] of its scale words
  __device__ __forceinline__ void scores(float (&s)[2][NH][4], const uint32_t (&kc)[2],
                                         const uint32_t (&ks)[2]) {
    const int gid = (threadIdx.x & 31) >> 2;
    // bytes e and e + 2 of the lane's scale words: its tokens (rows gid, gid + 8)
    const uint32_t sel = (gid & 1) ? 0x7351u : 0x6240u;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t kw[2][KW], ksc[KW / 2];
      ld_part<D / 8>(kc[hf], kw[0]);
      ld_part<D / 8, D>(kc[hf], kw[1]);
      ld_part<D / 16>(ks[hf], ksc);
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
        s[hf][nh][0] = s[hf][nh][1] = s[hf][nh][2] = s[hf][nh][3] = 0.f;
      // f16 scale pairs: sa = row gid's groups, sb = row gid + 8's
      uint32_t sa, sb;
      e4m3x4_to_f16x2x2(prmt(ksc[0], ksc[KW / 2 - 1], sel), sa, sb);
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        uint32_t a[4], b[4];
        e2m1x8_to_f16x2(kw[0][w], a);
        e2m1x8_to_f16x2(kw[1][w], b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // 16 codes are two words
          a[i] = w < 2 ? hmul2_lo(a[i], sa) : hmul2_hi(a[i], sa);
          b[i] = w < 2 ? hmul2_lo(b[i], sb) : hmul2_hi(b[i], sb);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int nh = 0; nh < NH; ++nh)
            mma_16816<false>(s[hf][nh], a[2 * u], b[2 * u], a[2 * u + 1], b[2 * u + 1],
                             qb[nh][2 * w + u][0], qb[nh][2 * w + u][1]);
      }
    }
  }

  // Weights of the tile's scores, exp2(s - base) as B fragments pb (pl: what
  // their rounding to binary16 left), and their sums.
  // The base is the largest score less kShift when it is set and stays until a
  // weight would pass exp2(kShift + kLag), so most tiles need neither the
  // maximum over lanes nor a rescale of o: one vote says so.
  // kEdge: only the tokens of `live` (a bit each) get a weight.
  template <bool kEdge>
  __device__ __forceinline__ void weights(float (&s)[2][NH][4], uint32_t live,
                                          uint32_t (&pb)[2][NH][2], uint32_t (&pl)[2][NH][2]) {
    const int gid = (threadIdx.x & 31) >> 2;
    const int tok = 4 * (gid >> 1) + (gid & 1);
    float mx[NH][2], top = -INFINITY;
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[hf][nh][e] = fmaf(s[hf][nh][e], sl[nh][e & 1], -base[nh][e & 1]);
          if constexpr (kEdge) {
            const int t = 16 * hf + tok + (e >> 1) * 2;
            if (!((live >> t) & 1u)) s[hf][nh][e] = -INFINITY;
          }
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[nh][e] = fmaxf(max3f(s[0][nh][e], s[0][nh][2 + e], s[1][nh][e]), s[1][nh][2 + e]);
      }
      top = max3f(top, mx[nh][0], mx[nh][1]);
    }
    if (__any_sync(kFull, top > limit)) {
      bool set = true;
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = mx[nh][e];
          x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
          x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
          x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
          // without weights so far the base goes anywhere, else only up (a
          // second copy goes with its first)
          float sum = l[nh][e];
          if constexpr (kTwin) sum = __shfl_sync(kFull, sum, threadIdx.x & 29);
          const bool fresh = sum == 0.f;
          float d = x - kShift;
          if (x == -INFINITY || (!fresh && d < 0.f)) d = 0.f;
          set = set && (!fresh || x > -INFINITY);
          alpha[e] = fresh ? 1.f : ex2_approx(-d);
          base[nh][e] += d;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            s[hf][nh][e] -= d;
            s[hf][nh][2 + e] -= d;
          }
          l[nh][e] *= alpha[e];
          l[nh][2 + e] *= alpha[e];
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          o[nh][i][0] *= alpha[0];
          o[nh][i][1] *= alpha[1];
          o[nh][i][2] *= alpha[0];
          o[nh][i][3] *= alpha[1];
        }
      }
      limit = __all_sync(kFull, set) ? kShift + kLag : -INFINITY;
    }
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float p0 = ex2_approx(s[hf][nh][2 * r]), p1 = ex2_approx(s[hf][nh][2 * r + 1]);
          uint32_t pk = pack2<false>(p0, p1);
          if constexpr (kTwin) {
            // the heads' second copy is left with the rest
            const float2 f = unpack2<false>((threadIdx.x & 2) != 0 ? pk : 0u);
            pk = pack2<false>(p0 - f.x, p1 - f.y);
          }
          if constexpr (kPair) {
            const float2 f = unpack2<false>(pk);
            pl[hf][nh][r] = movmatrix_trans(pack2<false>(p0 - f.x, p1 - f.y));
          }
          pb[hf][nh][r] = movmatrix_trans(pk);
        }
        // their sums, by a row of ones: the weights as they are used
        constexpr uint32_t kOnes = 0x3c003c00u;
        mma_16816<false>(l[nh], kOnes, kOnes, kOnes, kOnes, pb[hf][nh][0], pb[hf][nh][1]);
        if constexpr (kPair)
          mma_16816<false>(l[nh], kOnes, kOnes, kOnes, kOnes, pl[hf][nh][0], pl[hf][nh][1]);
      }
  }

  // O^T += V^T P^T of a tile: vc[hf] is the shared address of this lane's codes
  // of the first of its four rows, D / 2 bytes apart, vs[hf] of their scales.
  // kEdge: the scales of tokens outside `live`, which have weight zero, are
  // cleared: they may be NaN codes.
  template <bool kEdge>
  __device__ __forceinline__ void values(const uint32_t (&pb)[2][NH][2],
                                         const uint32_t (&pl)[2][NH][2], uint32_t live,
                                         const uint32_t (&vc)[2], const uint32_t (&vs)[2]) {
    const int tig = threadIdx.x & 3;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t vw[4][VW], sc[1];
      ld_part<D / 16>(vc[hf], vw[0]);
      ld_part<D / 16, D / 2>(vc[hf], vw[1]);
      ld_part<D / 16, D>(vc[hf], vw[2]);
      ld_part<D / 16, 3 * D / 2>(vc[hf], vw[3]);
      ld_part<4>(vs[hf], sc);
      if constexpr (kEdge) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (!((live >> (16 * hf + 4 * tig + b)) & 1u)) sc[0] &= ~(0xffu << (8 * b));
      }
      uint32_t s01, s23;
      e4m3x4_to_f16x2x2(sc[0], s01, s23);
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        const uint32_t v0 = vw[0][w], v1 = vw[1][w], v2 = vw[2][w], v3 = vw[3][w];
        constexpr uint32_t kLow = 0x0f0f0f0fu;
        // bytes of two tokens' codes of one head_dim: even and odd elements
        uint32_t a0[4], a1[4], a2[4], a3[4];
        e2m1x8_to_f16x2((v0 & kLow) | ((v1 << 4) & ~kLow), a0);
        e2m1x8_to_f16x2(((v0 >> 4) & kLow) | (v1 & ~kLow), a1);
        e2m1x8_to_f16x2((v2 & kLow) | ((v3 << 4) & ~kLow), a2);
        e2m1x8_to_f16x2(((v2 >> 4) & kLow) | (v3 & ~kLow), a3);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t x0 = hmul2(a0[b], s01), x1 = hmul2(a1[b], s01);
          const uint32_t x2 = hmul2(a2[b], s23), x3 = hmul2(a3[b], s23);
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) {
            mma_16816<false>(o[nh][4 * w + b], x0, x1, x2, x3, pb[hf][nh][0], pb[hf][nh][1]);
            if constexpr (kPair)
              mma_16816<false>(o[nh][4 * w + b], x0, x1, x2, x3, pl[hf][nh][0], pl[hf][nh][1]);
          }
        }
      }
    }
  }

  // the end of a context, or of a part: the heads' two copies become one
  __device__ __forceinline__ void finish() {
    if constexpr (kTwin) {
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
        for (int e = 0; e < 2; ++e) l[nh][e] += __shfl_xor_sync(kFull, l[nh][e], 2);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nh][i][e] += __shfl_xor_sync(kFull, o[nh][i][e], 2);
      }
    }
  }

  // the whole context: its output rows
  __device__ __forceinline__ void write(uint16_t* out, int G, float v_scale) const {
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float lt = l[nh][e];
        const int h = 8 * nh + 2 * tig + e;
        if (h >= G) continue;
        const float mul = lt == 0.f ? 0.f : v_scale / lt;
        uint4* dst = reinterpret_cast<uint4*>(out + (size_t)h * D + (D / 8) * gid);
#pragma unroll
        for (int i = 0; i < MT; i += 4) {
          uint4 pk;
          pk.x = pack2<kBF16>(o[nh][i][e] * mul, o[nh][i][2 + e] * mul);
          pk.y = pack2<kBF16>(o[nh][i + 1][e] * mul, o[nh][i + 1][2 + e] * mul);
          pk.z = pack2<kBF16>(o[nh][i + 2][e] * mul, o[nh][i + 2][2 + e] * mul);
          pk.w = pack2<kBF16>(o[nh][i + 3][e] * mul, o[nh][i + 3][2 + e] * mul);
          dst[i / 4] = pk;
        }
      }
  }

  // a part of it: o[G][D], m[G], l[G]
  __device__ __forceinline__ void store(float* rec, int G) const {
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float lt = l[nh][e];
        const int h = 8 * nh + 2 * tig + e;
        if (h >= G) continue;
        if (gid == 0) {
          rec[(size_t)G * D + h] = lt == 0.f ? -INFINITY : base[nh][e];
          rec[(size_t)G * D + G + h] = lt;
        }
        float4* dst = reinterpret_cast<float4*>(rec + (size_t)h * D + (D / 8) * gid);
#pragma unroll
        for (int i = 0; i < MT; i += 2)
          dst[i / 2] = make_float4(o[nh][i][e], o[nh][i][2 + e], o[nh][i + 1][e],
                                   o[nh][i + 1][2 + e]);
      }
  }
};

// Elements 4 c .. 4 c + 3 of row r of a record.
struct Vec {
  float4 o;
  float m, l;
  __device__ __forceinline__ void load(const float* rec, int G, int D, int r, int c) {
    o = *reinterpret_cast<const float4*>(rec + r * D + 4 * c);
    m = rec[G * D + r];
    l = rec[G * D + G + r];
  }
};

// Four elements of one row of a context, merged over parts: acc = sum_p
// 2^(m_p - m) o_p, l likewise, m the largest m_p.  The factors are ex2.approx: off
// by 2^-22, the same in o and l, below the weights' own rounding.
struct Merged {
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;

  __device__ __forceinline__ void fold(float mk, float lk, const float4& v) {
    const float mn = fmaxf(m, mk), base = mn == -INFINITY ? 0.f : mn;
    const float wa = ex2_approx(m - base), wb = ex2_approx(mk - base);
    m = mn;
    l = l * wa + lk * wb;
    acc.x = acc.x * wa + v.x * wb;
    acc.y = acc.y * wa + v.y * wb;
    acc.z = acc.z * wa + v.z * wb;
    acc.w = acc.w * wa + v.w * wb;
  }

  __device__ __forceinline__ void take_record(const float* rec, int G, int D, int r, int c) {
    Vec v;
    v.load(rec, G, D, r, c);
    acc = v.o;
    m = v.m;
    l = v.l;
  }
  __device__ __forceinline__ void fold_record(const float* rec, int G, int D, int r, int c) {
    Vec v;
    v.load(rec, G, D, r, c);
    fold(v.m, v.l, v.o);
  }
  __device__ __forceinline__ void store_record(float* rec, int G, int D, int r, int c) const {
    *reinterpret_cast<float4*>(rec + r * D + 4 * c) = acc;
    if (c == 0) {
      rec[G * D + r] = m;
      rec[G * D + G + r] = l;
    }
  }

  template <bool kBF16>
  __device__ __forceinline__ void write(uint16_t* dst, float v_scale) const {
    const float mul = l == 0.f ? 0.f : v_scale / l;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pack2<kBF16>(acc.x * mul, acc.y * mul), pack2<kBF16>(acc.z * mul, acc.w * mul));
  }
};

// A context's part held by one warp.
struct Part {
  long long pair;     // sequence * H + head, or -1
  long long g0;       // unit of the context's first tile
  int nt;             // its tiles
  int begins, ends;   // the part starts / ends with the context
  int rec;            // its record, in floats from the start of shared memory
};

// A context whose records, those of blocks first .. first + count - 1, are joined here.
struct Merge {
  long long pair;
  int first, count;
};

template <int kWarps>
struct Shared {
  long long run_pref[kWarps * 32];   // tiles (of one head) before each thread's run of sequences
  long long warp_tot[kWarps];
  int warp_longest[kWarps];
  Part part[2 * kWarps];
  int group_first[2 * kWarps + 1];
  int groups;
  int merges;                     // contexts this block owes the merge of
  Merge merge[2];
};

template <int D, bool kBF16, int NH, bool kTwin>
__global__ void __launch_bounds__(warps_of(NH) * 32, 1)
    decode_fp4_kernel(const Args a) {
  // per warp kStages tiles of K and V; after the last tile: [2 * kWarps] records
  extern __shared__ __align__(128) uint8_t dyn[];
  constexpr int kWarps = warps_of(NH), kThreads = 32 * kWarps;
  __shared__ Shared<kWarps> sh;
  constexpr int kRow = fp4_row_bytes(D), kPart = kTile * kRow, kStage = 2 * kPart;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const int B = 1 << a.log2B;
  const size_t rf = rec_floats(a.G, D);
  float* const slots = reinterpret_cast<float*>(dyn);

  // The small inputs towards L2 while the previous kernel in the stream drains
  // (a prefetch returns no data: that kernel may still be writing them).
  {
    const size_t step = (size_t)gridDim.x * kThreads * 128;
    const size_t at = ((size_t)blockIdx.x * kThreads + tid) * 128;
    const size_t sl_bytes = (size_t)a.num_seqs * 4, bt_bytes = sl_bytes * a.stride;
    const size_t q_bytes = (size_t)a.num_seqs * a.Hq * D * 2;
    for (size_t o = at; o < sl_bytes; o += step)
      prefetch_l2(reinterpret_cast<const char*>(a.seq_lens) + o);
    for (size_t o = at; o < bt_bytes; o += step)
      prefetch_l2(reinterpret_cast<const char*>(a.bt) + o);
    for (size_t o = at; o < q_bytes; o += step)
      prefetch_l2(reinterpret_cast<const char*>(a.q) + o);
  }
  if (!a.early_tables) grid_dep_wait();
  // ---- every thread counts the tiles of a run of sequences -----------------
  const int per = (a.num_seqs + kThreads - 1) / kThreads;
  const int run0 = min(a.num_seqs, tid * per), run1 = min(a.num_seqs, run0 + per);
  long long mine = 0;
  int longest = 0;
  bool odd = false;   // this block has to report or zero one of the run's sequences
  for (int i = run0; i < run1; ++i) {
    const int T = clamp_len(__ldg(a.seq_lens + i), a);
    // units, and above them the number of contexts that are not empty
    const int nt = num_tiles(T, a);
    longest = max(longest, nt);
    if (nt > 0) mine += nt + kStart + (i < kCounted ? 1ll << kUnitBits : 0ll);
    odd |= T == 0 && (i % gridDim.x) == blockIdx.x;
  }
  long long incl = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long n = __shfl_up_sync(kFull, incl, s);
    if (lane >= s) incl += n;
  }
  longest = __reduce_max_sync(kFull, longest);
  if (lane == 31) {
    sh.warp_tot[warp] = incl;
    sh.warp_longest[warp] = longest;
  }
  if (tid < 2 * kWarps) sh.part[tid].pair = -1;
  if (tid == 0) sh.merges = 0;
  __syncthreads();
  long long off = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) off += sh.warp_tot[w];
    total += sh.warp_tot[w];
    longest = max(longest, sh.warp_longest[w]);
  }
  // one context a warp (a unit is a context then)?
  const long long contexts = (total >> kUnitBits) * a.H;
  const bool whole = longest <= kWhole && a.num_seqs <= kCounted &&
                     contexts <= (long long)gridDim.x * kWarps;
  const long long low = (1ll << kUnitBits) - 1;
  const long long before = off + incl - mine;
  sh.run_pref[tid] = whole ? before >> kUnitBits : before & low;
  __syncthreads();
  if (a.early_tables) grid_dep_wait();
  if (tid == 0) grid_dep_launch();
  if (odd)
    for (int i = run0; i < run1; ++i) {
      if ((i % gridDim.x) != blockIdx.x) continue;
      const int T0 = __ldg(a.seq_lens + i);
      if (clamp_len(T0, a) != T0) set_error(a.err, PA_DEVERR_SEQ_LEN);
      if (clamp_len(T0, a) == 0) {
        uint4* dst = reinterpret_cast<uint4*>(a.out + (size_t)i * a.Hq * D);
        for (int e = 0; e < a.Hq * D / 8; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
      }
    }

  // ---- this block's and this warp's range of units -------------------------
  // about kLeast units a block in small batches, which then split contexts
  // between few blocks; whole, a context a warp
  const long long U = whole ? contexts : (total & low) * a.H;
  const int least = whole ? 1 : kLeast;
  const long long nb = min((long long)gridDim.x, (U + least - 1) / least);
  if ((long long)blockIdx.x >= nb) return;
  const long long c0 = U * blockIdx.x / nb, c1 = U * (blockIdx.x + 1) / nb;
  const long long n_cta = c1 - c0;
  // a warp's place in the block's range: neighbours on one scheduler (warp % 4),
  // so that few units fall on all four
  const int place = (warp & 3) * (kWarps / 4) + (warp >> 2);
  long long g = c0 + n_cta * place / kWarps;
  const long long g_end = c0 + n_cta * (place + 1) / kWarps;

  if (g < g_end) {
    // the sequence of unit g: the last run that starts at or before it, then
    // along the run
    int r = 0;
#pragma unroll
    for (int b = 256; b > 0; b >>= 1)
      if (r + b < kThreads && sh.run_pref[r + b] * a.H <= g) r += b;
    Walk w;   // the tile being computed
    w.i = r * per;
    w.load_seq(a);
    long long rem = g - sh.run_pref[r] * a.H;
    auto units = [&]() { return w.nt == 0 ? 0 : (whole ? 1 : w.nt + kStart); };   // of a head
    while (w.i < a.num_seqs && rem >= (long long)units() * a.H) {
      rem -= (long long)units() * a.H;
      ++w.i;
      w.load_seq(a);
    }
    const bool sound = w.i < a.num_seqs && rem >= 0;
    // only if seq_lens changes during the call (an error of the caller's): never
    // walk blind, here, at the next contexts or in the count of cut ones
    if (!sound) set_error(a.err, PA_DEVERR_SEQ_LEN);
    int left = 0;   // units to go, the tile's among them
    w.h = w.k = 0;
    if (sound) {
      w.h = (int)(rem / units());
      if (whole) {
        left = w.nt;
      } else {
        // a context's first kStart units are its start: the range begins with
        // its first tile, if it reaches that far.  g: the unit of the tile
        const int in_head = (int)(rem % units());
        w.k = max(0, in_head - kStart);
        g += w.k + kStart - in_head;
        if (g < g_end) left = (int)(g_end - g);
      }
    }
    int ld_left = left;

    // ---- the copies: K and V of a tile into stage n % kStages --------------
    // In shared memory a tile's K, and then its V, is a plane of bs = min(B, 32)
    // tokens, or several: codes, then scales.  Each of these is copied by its
    // own kLanes = bs lanes, 16 bytes a lane and copy: D / 32 copies of K and of
    // V, then the last bytes (the scales) of K by the first and of V by the next
    // D / 256 of the lanes.
    const uint32_t ring = smem_u32(dyn) + (uint32_t)(warp * kStages * kStage);
    Walk ld = w;
    const int bs = min(B, kTile), per_tile = kTile / bs;
    const int piece = lane / bs, u = lane & (bs - 1), last = bs * D / 256;
    const uint32_t block_bytes = (uint32_t)a.H * (uint32_t)a.plane;
    const bool last_k = u < last, last_v = !last_k && u < 2 * last;
    const uint32_t dst = ring + piece * (bs * kRow) + 16 * u;
    const uint32_t dst_last = ring + piece * (bs * kRow) + bs * (D / 2) +
                              (last_k ? 16 * u : 16 * (u - last) + kPart);
    const uint8_t* const pool_last =
        (last_k ? a.kc : a.vc) + (B * (D / 2) + 16 * (last_k ? u : u - last));
    int l_t0 = 0, l_last = 0, l_blk = 0;     // of the context being loaded
    uint32_t l_head = 0;                     // its head's plane in a block
    int win = -1, ent = -1;                  // entries [32 win, 32 win + 32) of its table row
    uint32_t win_bad = 0, bads = 0;          // those out of range; of the stages' blocks, 8 bits each
    auto load_context = [&]() {
      const int first = first_token(ld.T, a);
      l_blk = first >> a.log2B;
      l_t0 = (first / kTile + ld.k) * kTile;
      l_last = (ld.T - 1) >> a.log2B;
      l_head = (uint32_t)ld.h * (uint32_t)a.plane;
      win = -1;
    };
    load_context();
    auto issue = [&](int st) {
      const int blk0 = l_t0 >> a.log2B;
      if ((blk0 >> 5) != win) {
        win = blk0 >> 5;
        const int idx = 32 * win + lane;
        ent = -2;   // no entry
        // entries of blocks that hold an attended token
        if (idx >= l_blk && idx <= l_last) {
          ent = __ldg(a.bt + (size_t)ld.i * a.stride + idx);
          if (ent < 0 || (long long)ent >= a.num_blocks) {
            set_error(a.err, PA_DEVERR_BLOCK_ID);
            ent = -1;
          }
        }
        win_bad = __ballot_sync(kFull, ent == -1);
      }
      const uint32_t bad = (win_bad >> (blk0 & 31)) & ((1u << per_tile) - 1u);
      bads = (bads & ~(0xffu << (8 * st))) | (bad << (8 * st));
      const uint32_t tok = (uint32_t)l_t0 & (uint32_t)(B - 1);   // 0 but in larger blocks
      const uint32_t so = (uint32_t)(st * kStage);
      const int e = __shfl_sync(kFull, ent, blk0 + piece);
      if (e >= 0) {
        const uint64_t at = (uint64_t)(uint32_t)e * block_bytes + l_head;
        const uint64_t codes = at + (tok * (D / 2) + 16 * u);
        const uint8_t *k = a.kc + codes, *v = a.vc + codes;
        if (bs == 32) copy_codes<D, 32>(dst + so, k, v);
        else if (bs == 16) copy_codes<D, 16>(dst + so, k, v);
        else if (bs == 8) copy_codes<D, 8>(dst + so, k, v);
        else copy_codes<D, 4>(dst + so, k, v);
        if (last_k || last_v) copy16(dst_last + so, pool_last + (at + tok * (D / 16)));
      }
      l_t0 += kTile;
      --ld_left;
      if (++ld.k == ld.nt) {
        --ld.k;
        ld.advance(a);
        ld_left -= kStart;
        if (ld.nt > 0) load_context();
        else ld_left = 0;   // past the last sequence
      }
    };
    // this lane's bytes of a tile.  K: rows (gid & 1) and (gid & 1) + 2 of token
    // group gid / 2 of each half; V: the four of group tig.
    uint32_t ok[2], os[2], ov[2], ow[2];
    {
      const uint32_t pl_bytes = (uint32_t)(bs * kRow);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int tk = 16 * hf + 4 * (gid >> 1), tv = 16 * hf + 4 * tig;
        const int rk = tk & (bs - 1), rv = tv & (bs - 1);
        const uint32_t pk = (uint32_t)(tk / bs) * pl_bytes, pv = (uint32_t)(tv / bs) * pl_bytes;
        ok[hf] = ring + pk + (rk + (gid & 1)) * (D / 2) + tig * (D / 8);
        os[hf] = ring + pk + bs * (D / 2) + rk * (D / 16) + tig * (D / 16);
        ov[hf] = ring + kPart + pv + rv * (D / 2) + gid * (D / 16);
        ow[hf] = ring + kPart + pv + bs * (D / 2) + rv * (D / 16) + (D == 128 ? gid : gid >> 1) * 4;
      }
    }

    Context<D, kBF16, NH, kTwin> cx;
    for (int n = 0; n < kStages; ++n) {
      if (ld_left > 0) issue(n);
      copies_commit();   // of every tile, issued or not: one group each
    }
    int st = 0, segments = 0;
    while (left > 0) {
      // a context, or this warp's part of one: its tiles w.k .. w.k + run - 1
      const int run = min(w.nt - w.k, left), first = first_token(w.T, a);
      const bool ends = w.k + run == w.nt;
      g -= w.k;   // the unit of its first tile
      cx.begin(a.q + ((size_t)w.i * a.Hq + (size_t)w.h * a.G) * D, a.G, a.scale_log2);
      int t0 = (first / kTile + w.k) * kTile;
      for (int n = run; n > 0; --n) {
        copies_wait<kStages - 1>();
        __syncwarp();   // every lane's copies of this tile have landed
        const uint32_t so = (uint32_t)(st * kStage);
        const uint32_t bad = (bads >> (8 * st)) & 0xffu;
        const bool edge = t0 < first || w.T - t0 < kTile || bad != 0u;
        float s[2][NH][4];
        uint32_t pb[2][NH][2], pl[2][NH][2];
        const uint32_t kc[2] = {ok[0] + so, ok[1] + so}, ks[2] = {os[0] + so, os[1] + so};
        const uint32_t vc[2] = {ov[0] + so, ov[1] + so}, vs[2] = {ow[0] + so, ow[1] + so};
        cx.scores(s, kc, ks);
        if (edge) {
          uint32_t live = kFull;
          if (t0 < first) live &= kFull << (first - t0);
          if (w.T - t0 < kTile) live &= kFull >> (kTile - (w.T - t0));
          if (bad)
            for (int b = 0; b < kTile / bs; ++b)
              if ((bad >> b) & 1u) live &= ~((bs == 32 ? kFull : (1u << bs) - 1u) << (b * bs));
          cx.template weights<true>(s, live, pb, pl);
          cx.template values<true>(pb, pl, live, vc, vs);
        } else {
          cx.template weights<false>(s, kFull, pb, pl);
          cx.template values<false>(pb, pl, kFull, vc, vs);
        }
        __syncwarp();   // every lane has read the stage
        if (ld_left > 0) issue(st);
        copies_commit();
        if (++st == kStages) st = 0;
        t0 += kTile;
      }
      left -= run;
      // the end of the context, or of this warp's part of it.  The warp's last
      // part goes where its tiles were, an earlier one to the warp's slot.
      cx.finish();
      if (w.k == 0 && ends) {
        cx.write(a.out + ((size_t)w.i * a.Hq + (size_t)w.h * a.G) * D, a.G, a.v_scale);
      } else {
        const int rec = left <= (ends ? kStart : 0)
                            ? warp * (kStages * kStage / 4)
                            : kWarps * (kStages * kStage / 4) + warp * (int)rf;
        cx.store(slots + rec, a.G);
        if (lane == 0) {
          Part& p = sh.part[2 * place + (segments > 0 ? 1 : 0)];
          p.pair = (long long)w.i * a.H + w.h;
          p.g0 = g;
          p.nt = w.nt;
          p.begins = w.k == 0;
          p.ends = ends;
          p.rec = rec;
        }
      }
      ++segments;
      // the next context of the range, if there is one
      g += w.nt + kStart;
      left -= kStart;
      w.k = w.nt - 1;
      if (left > 0) w.advance(a);
      if (left > 0 && w.nt == 0) {   // past the last sequence: not blind either
        set_error(a.err, PA_DEVERR_SEQ_LEN);
        left = 0;
      }
    }
    copies_wait<0>();   // none, unless the loads' walk met other lengths
  }
  __syncthreads();

  // ---- parts of one context held by this block's warps ---------------------
  // parts are in tile order; those of one context follow each other
  if (warp == 0) {
    const bool held = lane < 2 * kWarps && sh.part[lane].pair >= 0;
    const uint32_t all = __ballot_sync(kFull, held);
    const uint32_t before = all & ((1u << lane) - 1u);
    const bool starts =
        held && (before == 0u || sh.part[31 - __clz(before)].pair != sh.part[lane].pair);
    const uint32_t firsts = __ballot_sync(kFull, starts);
    if (starts) sh.group_first[__popc(firsts & ((1u << lane) - 1u))] = lane;
    if (lane == 0) {
      sh.groups = __popc(firsts);
      sh.group_first[__popc(firsts)] = 2 * kWarps;
    }
  }
  __syncthreads();
  constexpr int cols = D / 4;
  const int per_group = a.G * cols;
  const int step_gr = kThreads / per_group, step_t = kThreads % per_group;
  for (int gr = tid / per_group, t = tid % per_group; gr < sh.groups;) {
    const int r = t / cols, c = t % cols;
    const int k0 = sh.group_first[gr], k1 = sh.group_first[gr + 1];
    const long long pair = sh.part[k0].pair;
    const int begins = sh.part[k0].begins;
    int ends = sh.part[k0].ends;
    Merged x;
    x.take_record(slots + sh.part[k0].rec, a.G, D, r, c);
    for (int k = k0 + 1; k < k1; ++k) {
      if (sh.part[k].pair < 0) continue;
      ends = sh.part[k].ends;
      x.fold_record(slots + sh.part[k].rec, a.G, D, r, c);
    }
    if (begins && ends)
      x.write<kBF16>(a.out + ((size_t)pair * a.G + r) * D + 4 * c, a.v_scale);
    else   // record 0: the context began in an earlier block; 1: it begins here
      x.store_record(a.ws_rec + ((size_t)blockIdx.x * 2 + begins) * rf, a.G, D, r, c);
    gr += step_gr;
    t += step_t;
    if (t >= per_group) {
      t -= per_group;
      ++gr;
    }
  }
  __syncthreads();
  // ---- contexts cut between blocks: count this block's record --------------
  if (tid < sh.groups) {
    const Part p = sh.part[sh.group_first[tid]];
    if (p.g0 < c0 || p.g0 + p.nt > c1) {   // else inside this block's range: already written
      const long long f = ((p.g0 + 1) * nb - 1) / U, e = ((p.g0 + p.nt) * nb - 1) / U;
      uint32_t* cnt = a.ws_count + e;
      // a block's first and last context alone may be cut, and it lies among the
      // blocks that hold them, unless seq_lens changed during the call
      const bool cut = (tid == 0 || tid == sh.groups - 1) && f >= 0 && f <= blockIdx.x &&
                       e >= blockIdx.x && e < nb;
      if (!cut) set_error(a.err, PA_DEVERR_SEQ_LEN);
      // releases the block's record (ordered before by the barrier), acquires
      // those counted before it
      if (cut && atom_add_acq_rel_gpu(cnt, 1u) + 1u == (uint32_t)(e - f + 1)) {
        *cnt = 0u;   // ready for the next call
        Merge& m = sh.merge[atomicAdd(&sh.merges, 1)];
        m.pair = p.pair;
        m.first = (int)f;
        m.count = (int)(e - f + 1);
      }
    }
  }
  __syncthreads();
  // ---- the contexts whose last record this block counted -------------------
  // their records, record 1 of the first block and record 0 of the others, in
  // equal runs over the threads that a context's vectors leave free
  for (int k = 0; k < sh.merges; ++k) {
    const Merge m = sh.merge[k];
    const float* const recs = a.ws_rec + (size_t)m.first * 2 * rf;
    uint16_t* const out = a.out + (size_t)m.pair * a.G * D;
    const int rows = per_group, runs = m.count <= kRecords ? 1 : max(1, kThreads / rows);
    const int run = runs == 1 ? 0 : tid / rows;
    for (int t = tid - run * rows; t < rows && run < runs; t += kThreads) {
      const int r = t / cols, c = t % cols;
      const int n1 = m.count * (run + 1) / runs;
      Merged x;
      for (int n = m.count * run / runs; n < n1; n += kRecords) {
        Vec v[kRecords];
#pragma unroll
        for (int b = 0; b < kRecords; ++b) {
          const int i = min(n + b, n1 - 1);
          v[b].load(recs + (size_t)(2 * i + (i == 0 ? 1 : 0)) * rf, a.G, D, r, c);
        }
#pragma unroll
        for (int b = 0; b < kRecords; ++b)
          if (n + b < n1) x.fold(v[b].m, v[b].l, v[b].o);
      }
      if (runs == 1)
        x.write<kBF16>(out + (size_t)4 * t, a.v_scale);
      else
        x.store_record(slots + run * rf, a.G, D, r, c);
    }
    if (runs > 1) {
      __syncthreads();
      if (tid < rows) {
        Merged x;
        for (int b = 0; b < runs; ++b) x.fold_record(slots + b * rf, a.G, D, tid / cols, tid % cols);
        x.write<kBF16>(out + (size_t)4 * tid, a.v_scale);
      }
      __syncthreads();
    }
  }
}

typedef void (*Kernel)(const Args);

template <int D>
Kernel pick_d(bool bf16, int G) {
  if (bf16)
    return G > 8 ? decode_fp4_kernel<D, true, 2, false>
                 : (G > 4 ? decode_fp4_kernel<D, true, 1, false> : decode_fp4_kernel<D, true, 1, true>);
  return G > 8 ? decode_fp4_kernel<D, false, 2, false>
               : (G > 4 ? decode_fp4_kernel<D, false, 1, false> : decode_fp4_kernel<D, false, 1, true>);
}

// the ring of every warp (which its last part's record shares) and a slot each
// for an earlier part
size_t smem_bytes(int D, int G) {
  return (size_t)warps_of(G > 8 ? 2 : 1) *
         (kStages * 2 * kTile * fp4_row_bytes(D) + rec_floats(G, D) * sizeof(float));
}
static_assert(rec_floats(16, 128) * 4 <= kStages * 2 * kTile * fp4_row_bytes(128) &&
                  rec_floats(16, 64) * 4 <= kStages * 2 * kTile * fp4_row_bytes(64),
              "a record fits in a warp's ring");

struct Plan {
  Kernel kern;
  int grid, threads;
  size_t smem, count_bytes, rec_bytes;
};

// The kernels' opt-in to their shared memory, once a device.
constexpr int kMaxDevices = 64;
bool g_ready[kMaxDevices][2][2][3];   // [device][D == 128][bf16][heads <= 4, <= 8, <= 16]
std::mutex g_mu;

int make_plan(int Hq, int H, int D, int B, int q_dtype, int flags, int num_ctas, Plan* p) {
  if (Hq <= 0 || H <= 0 || num_ctas < 0 || num_ctas > PA_DECODE_MAX_CTAS)
    return PA_ERR_INVALID_ARG;
  if (q_dtype != PA_F16 && q_dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (D != 64 && D != 128) return PA_ERR_UNSUPPORTED;
  if (!is_pow2(B) || B < 4 || B > 256) return PA_ERR_UNSUPPORTED;
  if (Hq % H != 0) return PA_ERR_INVALID_ARG;
  const int G = Hq / H;
  if (G > 16) return PA_ERR_UNSUPPORTED;
  // a block's bytes are counted in 31 bits
  if ((long long)H * B * fp4_row_bytes(D) > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
  flags &= ~PA_DECODE_TABLES_READY;
  if (flags == PA_DECODE_SIMT) return PA_ERR_UNSUPPORTED;
  if (flags != PA_DECODE_AUTO && flags != PA_DECODE_MMA) return PA_ERR_INVALID_ARG;
  const bool bf16 = q_dtype == PA_BF16;
  p->kern = D == 64 ? pick_d<64>(bf16, G) : pick_d<128>(bf16, G);
  p->smem = smem_bytes(D, G);
  DeviceInfo di;
  if (int rc = current_device_info(&di)) return rc;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    bool& ready = g_ready[di.device][D == 128][bf16][G > 8 ? 2 : (G > 4 ? 1 : 0)];
    if (!ready) {
      const cudaError_t e =
          cudaFuncSetAttribute(p->kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)smem_bytes(D, G > 8 ? 16 : 8));
      if (e) return launch_status(e, "cudaFuncSetAttribute (4-bit decode)");
      ready = true;
    }
  }
  p->threads = 32 * warps_of(G > 8 ? 2 : 1);
  p->grid = num_ctas > 0 ? num_ctas : di.sm_count;
  if (p->grid > PA_DECODE_MAX_CTAS) return PA_ERR_INVALID_ARG;
  p->count_bytes = (size_t)PA_DECODE_MAX_CTAS * sizeof(uint32_t);
  p->rec_bytes = (size_t)p->grid * 2 * rec_floats(G, D) * sizeof(float);
  return PA_OK;
}

}  // namespace

int decode_fp4_workspace(int Hq, int H, int D, int B, int flags, int num_ctas, size_t* bytes) {
  Plan b{}, f{};
  // the larger of the two query dtypes' grids
  if (int rc = make_plan(Hq, H, D, B, PA_BF16, flags, num_ctas, &b)) return rc;
  if (int rc = make_plan(Hq, H, D, B, PA_F16, flags, num_ctas, &f)) return rc;
  *bytes = b.count_bytes + (b.rec_bytes > f.rec_bytes ? b.rec_bytes : f.rec_bytes);
  return PA_OK;
}

}  // namespace pa

using namespace pa;

extern "C" int pa_decode_fp4(const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_tables, int32_t table_stride,
                             const int32_t* seq_lens, int32_t num_seqs, int32_t num_q_heads,
                             int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                             int64_t num_blocks, int32_t q_dtype, float scale, float k_scale,
                             float v_scale, int32_t window, void* out, void* workspace,
                             size_t workspace_bytes, int32_t flags, int32_t num_ctas,
                             int32_t* err_word, pa_stream stream) {
  if (num_seqs < 0 || table_stride < 0 || num_blocks < 0 || window < 0) return PA_ERR_INVALID_ARG;
  if (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
    return PA_ERR_INVALID_ARG;
  Plan p{};
  if (int rc = make_plan(num_q_heads, num_kv_heads, head_dim, block_size, q_dtype, flags, num_ctas,
                         &p))
    return rc;
  if (num_seqs == 0) return PA_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !out || !workspace)
    return PA_ERR_INVALID_ARG;
  if (num_blocks == 0 || table_stride == 0) return PA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned16(workspace))
    return PA_ERR_INVALID_ARG;
  if (workspace_bytes < p.count_bytes + p.rec_bytes) return PA_ERR_WORKSPACE;
  Args a{};
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.kc = static_cast<const uint8_t*>(k_cache);
  a.vc = static_cast<const uint8_t*>(v_cache);
  a.bt = block_tables;
  a.seq_lens = seq_lens;
  a.ws_count = static_cast<uint32_t*>(workspace);
  a.ws_rec = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.count_bytes);
  a.err = err_word;
  a.num_blocks = num_blocks;
  a.num_seqs = num_seqs;
  a.stride = table_stride;
  a.Hq = num_q_heads;
  a.H = num_kv_heads;
  a.G = num_q_heads / num_kv_heads;
  a.log2B = ilog2(block_size);
  a.plane = block_size * fp4_row_bytes(head_dim);
  a.scale_log2 = scale * k_scale * 1.4426950408889634f;
  a.v_scale = v_scale;
  a.window = window;
  a.early_tables = (flags & PA_DECODE_TABLES_READY) ? 1 : 0;
  clear_stale_error();
  return launch_status(launch_pdl(p.kern, dim3((unsigned)p.grid), dim3((unsigned)p.threads), p.smem,
                                  static_cast<cudaStream_t>(stream), a),
                       "4-bit decode launch");
}
