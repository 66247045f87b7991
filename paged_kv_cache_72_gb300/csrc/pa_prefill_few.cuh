// Chunks of few rows: attention of sequences whose new tokens make at most kFewRows
// query rows (tokens times query heads of a KV head) over quantized KV caches, the
// formulas of pa_prefill_quant.cuh.
//
// Bound: bytes; the tensor-memory kernel, whose tiles have 128 rows, spends some
// 1,700 cycles on 64 keys whatever their rows.  Here the rows are the narrow side of
// warp-level products: S^T = K Q^T (16 keys x 8 rows) and O^T += V^T P^T (16 head_dim
// rows x 8 rows), so that a tile of 32 keys is converted once, in registers, and
// used for one or two columns of 8 rows.  The rate of these products ends its use:
// with four columns 32 rows took 1,000 us where the other kernel takes 597.
//
// Measured, 32 contexts of 16 to 33 K tokens, 64 query and 8 KV heads of 128 (the other
// kernel: 600 us each): one new token 305 us over E4M3 (5.4 TB/s), 285 over 4 bits (3.3
// TB/s: the conversion's instructions and their latencies with 8 warps an SM), two
// tokens 332 and 316.  For rows of one column alone 16 warps an SM took 288 and 223 us,
// but two tokens then 608.
//
// The weights are one binary16 value each (2^-11), as in the other kernel, so that a
// call's rows are alike: binary16 outputs are 2.8e-4 off 64 bits in norm (2.1e-4 is their
// own rounding), bfloat16 ones 1.7e-3 with either.  A pair of values, as the 4-bit decode
// has, takes second products: one token 336 us over E4M3 and 325 over 4 bits, two 372 and 371.
//
//  * The tiles of all (sequence, KV head) contexts are a line, kStartTiles and one
//    for each tile a context, cut into equal shares, one a block.  The warps
//    of a block take the tiles of its part of a context in turn, each through a ring
//    of its own (16-byte asynchronous copies), join their partial results in shared
//    memory, and write the rows, or a record where the context is cut between
//    blocks; the last block to count its record joins them, in the order of the keys.
//    Two blocks of four warps an SM, so that one computes while the other starts or
//    ends a context: 512 contexts of 1 K tokens took 46 us, in blocks of eight warps
//    59, of twelve 71.
//  * Index maps as in the 4-bit decode: MMA row r < 8 of a half tile is token 4 (r /
//    2) + r % 2, row 8 + r the token two further; S^T's k index 2 tig + e of step s
//    is head_dim (D / 4) tig + 4 s + e, and 8 + 2 tig + e two further; O^T's row gid
//    of m-tile i is (D / 8) gid + 2 i, row 8 + gid the next.
#pragma once

namespace pa {

namespace {

constexpr int kFewWarps = 4;
constexpr int kFewBlocks = 2;        // an SM
constexpr int kFewThreads = 32 * kFewWarps;
constexpr int kTile = 32;            // keys
constexpr int kStartTiles = 8;       // what a context's start and end cost, in tiles
constexpr int kLeastTiles = 16;      // of the line, a block's in small batches
constexpr int kColumns = kFewRows / 8;
constexpr uint32_t kAll = 0xffffffffu;

__host__ __device__ constexpr size_t few_rec_floats(int D) { return (size_t)kFewRows * (D + 2); }

// A tile in shared memory: K, then V: 32 rows of codes, then a 4-bit pool's scales,
// eight quads of D / 4 bytes.  16-byte chunk c of row r lies at c ^ swizzle(r), which
// keeps the reads of a warp's eight neighbours in different banks.
template <int D, bool kFour>
struct FewTile {
  static constexpr int kRowBytes = kFour ? D / 2 : D;
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kCodes = kTile * kRowBytes;
  static constexpr int kHalf = kCodes + (kFour ? 2 * D : 0);
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = kFour ? 4 : 3;
  static constexpr int kCopies = kCodes / 512;    // a lane's of K, and of V
  __device__ static __forceinline__ int swizzle(int r) {
    return (kChunks == 8 ? (((r >> 2) & 3) << 1) | (r & 1) : (r >> 2)) & (kChunks - 1);
  }
};

// A context: a sequence and KV head, and its place on the line.
struct FewContext {
  int i, q0, L, T, first, nt, h;
  long long i0;
};

template <int D, bool kFour>
struct FewShared {
  uint2 q[D / 16][kColumns][32];     // query fragments
  float factor[kFewRows];            // what a row's scores are multiplied by
  int pos[kFewRows];                 // its position, -1: no row
  long long run_pref[kFewThreads];
  long long warp_tot[kFewWarps];
  long long bound[kFewBlocks * kMaxGrid + 1];
  uint16_t parts[kFewBlocks * kMaxGrid];
  int nparts, last;
  FewContext context[2];             // this one and the next, in turn
  float ml[kFewWarps][2][kFewRows];
  float join[kFewRows][2];
  int bad[kFewRows];                 // a NaN among the row's sums
  // the rings; at a context's end the warps' sums, [warp][row][D]
  static constexpr size_t kRings =
      (size_t)kFewWarps * FewTile<D, kFour>::kStages * FewTile<D, kFour>::kStage;
  static constexpr size_t kSums = (size_t)kFewWarps * kFewRows * D * sizeof(float);
  alignas(128) uint8_t data[kRings > kSums ? kRings : kSums];
};

// A sequence's tiles of one KV head: from the one with its first attended token; 0
// where it has no new tokens or more rows than are dealt with here.
__device__ __forceinline__ int few_tiles(const Args& a, int i, int& q0, int& L, int& T,
                                         int& first) {
  load_any(a, i, q0, L, T);
  first = 0;
  if (L == 0 || (long long)L * a.G > kFewRows) return 0;
  const long long f = (long long)T - L - a.window + 1;
  if (a.window > 0 && f > 0) first = (int)f;
  return (T - 1) / kTile - first / kTile + 1;
}

template <int D, bool kBF16, bool kFour>
__global__ void __launch_bounds__(kFewThreads, kFewBlocks) prefill_few_kernel(const Args a) {
  using X = FewTile<D, kFour>;
  extern __shared__ __align__(128) uint8_t few_raw[];
  FewShared<D, kFour>& c = *reinterpret_cast<FewShared<D, kFour>*>(few_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const int B = 1 << a.log2B;
  grid_dep_wait();

  // ---- the line: every thread sums a run of sequences ----------------------
  const int per = (a.num_seqs + kFewThreads - 1) / kFewThreads;
  const int run0 = min(a.num_seqs, tid * per), run1 = min(a.num_seqs, run0 + per);
  int q0 = 0, L = 0, T = 0, first = 0;
  long long mine = 0;
  bool odd = false;
  for (int i = run0; i < run1; ++i) {
    odd |= !load_any(a, i, q0, L, T);
    const int nt = few_tiles(a, i, q0, L, T, first);
    if (nt > 0) mine += (long long)(nt + kStartTiles) * a.H;
  }
  long long incl = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long n = __shfl_up_sync(kAll, incl, s);
    if (lane >= s) incl += n;
  }
  if (lane == 31) c.warp_tot[warp] = incl;
  odd = __syncthreads_or(odd && a.few == kFewOnly) != 0;
  long long off = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kFewWarps; ++w) {
    if (w < warp) off += c.warp_tot[w];
    total += c.warp_tot[w];
  }
  c.run_pref[tid] = off + incl - mine;
  if (tid == 0) grid_dep_launch();
  if (odd) clear_bad(a, D, kFewThreads);
  const long long nb = min((long long)gridDim.x, (total + kLeastTiles - 1) / kLeastTiles);
  if ((long long)blockIdx.x >= nb) return;
  for (int k = tid; k <= nb; k += kFewThreads) c.bound[k] = total * k / nb;
  __syncthreads();
  const long long u0 = c.bound[blockIdx.x], u1 = c.bound[blockIdx.x + 1];

  // ---- the context at place u0.  One thread walks and the block takes what it found:
  // lengths that change during the call then cannot part the block's threads.
  if (tid == 0) {
    FewContext x{};
    int r = 0;   // the last run that starts at or before u0
#pragma unroll
    for (int b = 256; b > 0; b >>= 1)
      if (r + b < kFewThreads && c.run_pref[r + b] <= u0) r += b;
    x.i = r * per;
    x.i0 = c.run_pref[r];
    while (x.i < a.num_seqs) {
      x.nt = few_tiles(a, x.i, x.q0, x.L, x.T, x.first);
      const long long one = x.nt > 0 ? (long long)(x.nt + kStartTiles) * a.H : 0;
      if (u0 < x.i0 + one) break;
      x.i0 += one;
      ++x.i;
    }
    if (x.i < a.num_seqs) {
      x.h = (int)((u0 - x.i0) / (x.nt + kStartTiles));
      x.i0 += (long long)x.h * (x.nt + kStartTiles);
    }
    c.context[0] = x;
  }
  __syncthreads();
  int turn = 0, i = 0, h = 0, nt = 0;
  long long i0 = 0;
  auto take = [&]() {
    const FewContext& x = c.context[turn];
    i = x.i;
    q0 = x.q0;
    L = x.L;
    T = x.T;
    first = x.first;
    nt = x.nt;
    h = x.h;
    i0 = x.i0;
  };
  take();
  // The next context, by thread 0, once a turn of the loop below, before a barrier of it:
  // the block takes it behind that one, and is done with the other place before it.
  auto walk_on = [&]() {
    if (tid != 0) return;
    FewContext x = c.context[turn];
    x.i0 += x.nt + kStartTiles;
    if (++x.h == a.H) {
      x.h = 0;
      x.nt = 0;
      while (x.nt == 0 && ++x.i < a.num_seqs)
        x.nt = few_tiles(a, x.i, x.q0, x.L, x.T, x.first);
    }
    c.context[turn ^ 1] = x;
  };
  const uint32_t ring = smem_u32(c.data) + (uint32_t)(warp * X::kStages * X::kStage);
  const size_t block_bytes = kFour ? (size_t)a.H * B * fp4_row_bytes(D) : (size_t)B * a.H * D;

  while (i < a.num_seqs && i0 < u1) {
    // this block's tiles of the context: those that stand in its share
    auto tile_at = [&](long long at) -> int {
      const long long k = at - i0 - kStartTiles;
      return k <= 0 ? 0 : (k < nt ? (int)k : nt);
    };
    const int k0 = tile_at(u0), k1 = tile_at(u1);
    if (k0 < k1) {
      const int rows = L * a.G, cols = (rows + 7) >> 3;
      // ---- the query rows as f16 fragments, eight threads a row.  A bfloat16 row is
      // brought into binary16's range by a power of two (its largest magnitude into
      // [1, 2)), which its score factor takes back.
      {
        constexpr int kWordsQ = D / 16;          // of a thread's D / 8 elements
        const int r = tid >> 3, t8 = tid & 7;
        uint32_t y[kWordsQ];
        const int tok = r / a.G;
#pragma unroll
        for (int v = 0; v < kWordsQ / 4; ++v) {
          uint4 z = make_uint4(0u, 0u, 0u, 0u);
          if (r < rows)
            z = __ldg(reinterpret_cast<const uint4*>(
                    a.q + ((size_t)(q0 + tok) * a.Hq + (size_t)h * a.G + (r - tok * a.G)) * D +
                    (D / 8) * t8) + v);
          y[4 * v] = z.x; y[4 * v + 1] = z.y; y[4 * v + 2] = z.z; y[4 * v + 3] = z.w;
        }
        float back = 1.f;
        if constexpr (kBF16) {
          float mx = 0.f;
#pragma unroll
          for (int v = 0; v < kWordsQ; ++v) {
            const float2 f = unpack2<true>(y[v]);
            mx = max3f(mx, fabsf(f.x), fabsf(f.y));
          }
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2));
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 4));
          const int e = min(max((int)(__float_as_uint(mx) >> 23), 1), 253);
          back = __uint_as_float((uint32_t)e << 23);
          const float to = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
          for (int v = 0; v < kWordsQ; ++v) {
            const float2 f = unpack2<true>(y[v]);
            y[v] = pack2<false>(f.x * to, f.y * to);
          }
        }
        // head_dim (D / 8) t8 + 4 v .. + 3: step s of the lanes with tig = t8 / 2
        if (r < kFewRows) {
#pragma unroll
          for (int v = 0; v < kWordsQ / 2; ++v)
            c.q[(t8 & 1) * (D / 32) + v][r >> 3][4 * (r & 7) + (t8 >> 1)] =
                make_uint2(y[2 * v], y[2 * v + 1]);
        }
        if (t8 == 0 && r < kFewRows) {
          c.factor[r] = a.scale_log2 * back;
          c.pos[r] = r < rows ? T - L + tok : -1;
          c.bad[r] = 0;
        }
      }
      // ---- this warp's tiles: k0 + warp, every fourth
      // lane j: the j-th block of tile k, and whether a row of it is attended to (apart from
      // the entry, which may hold anything and is not waited for here)
      bool need = false;
      auto entries = [&](int k) -> int {
        const int t0 = (int)((uint32_t)(first / kTile + k) * kTile);   // (k < k1: in range)
        const int idx = (t0 >> a.log2B) + lane;
        need = k < k1 && lane < max(kTile >> a.log2B, 1) && idx >= (first >> a.log2B) &&
               idx <= ((T - 1) >> a.log2B);
        return need ? __ldg(a.bt + (size_t)i * a.stride + idx) : -1;
      };
      uint32_t missing = 0u;   // a bit a ring slot: some row's block is not there
      uint32_t bads[X::kStages];   // rows whose block is out of range
      int next = k0 + warp, ent = entries(next);
      auto issue = [&](int slot) {
        const int t0 = (first / kTile + next) * kTile;
        const bool bad = need && (ent < 0 || (long long)ent >= a.num_blocks);
        if (bad) {
          set_error(a.err, PA_DEVERR_BLOCK_ID);
          ent = -1;
        }
        const int nblk = max(kTile >> a.log2B, 1), bs = min(B, kTile);
        const uint32_t gone = __ballot_sync(kAll, ent < 0) & (kAll >> (32 - nblk));
        uint32_t rows_bad = __ballot_sync(kAll, bad);
        missing = (missing & ~(1u << slot)) | (gone ? 1u << slot : 0u);
        uint32_t wide = 0u;
        for (int b = 0; rows_bad >> b; ++b)
          if ((rows_bad >> b) & 1u) wide |= (kAll >> (32 - bs)) << (b * bs);
#pragma unroll
        for (int k = 0; k < X::kStages; ++k)
          if (k == slot) bads[k] = wide;
        const uint32_t dst = ring + (uint32_t)(slot * X::kStage);
#pragma unroll
        for (int k = 0; k < X::kCopies; ++k) {
          const int p = lane + 32 * k, r = p / X::kChunks, ch = p % X::kChunks;
          const int e = __shfl_sync(kAll, ent, r >> min(a.log2B, 5));
          const int rb = (t0 + r) & (B - 1);
          if (e >= 0) {
            const size_t at =
                kFour ? e * block_bytes + (size_t)h * (B * fp4_row_bytes(D)) + rb * (D / 2) + 16 * ch
                      : e * block_bytes + ((size_t)rb * a.H + h) * D + 16 * ch;
            const uint32_t to = dst + (uint32_t)(r * X::kRowBytes + ((ch ^ X::swizzle(r)) << 4));
            copy16(to, a.kc + at);
            copy16(to + X::kHalf, a.vc + at);
          }
        }
        if constexpr (kFour) {   // the quads' scales: K's by the first lanes, then V's
          constexpr int kPer = D / 64, kLanes = 8 * kPer;
          const int p = lane % kLanes, r = 4 * (p / kPer);
          const int e = __shfl_sync(kAll, ent, r >> min(a.log2B, 5));
          const int rb = (t0 + r) & (B - 1);
          if (e >= 0 && lane < 2 * kLanes)
            copy16(dst + (uint32_t)(X::kCodes + 16 * p + (lane < kLanes ? 0 : X::kHalf)),
                   (lane < kLanes ? a.kc : a.vc) + e * block_bytes +
                       (size_t)h * (B * fp4_row_bytes(D)) + B * (D / 2) + rb * (D / 16) +
                       16 * (p % kPer));
        }
        next += kFewWarps;
        ent = entries(next);
      };
#pragma unroll
      for (int k = 0; k < X::kStages; ++k) {
        bads[k] = 0u;
        if (next < k1) issue(k);
        commit_copies();
      }
      walk_on();
      __syncthreads();   // the fragments, factors and positions
      float o[kColumns][D / 16][4], l[kColumns][4], base[kColumns][2], sl[kColumns][2];
      bool poison[kColumns][2];
#pragma unroll
      for (int n = 0; n < kColumns; ++n) {
#pragma unroll
        for (int m = 0; m < D / 16; ++m) o[n][m][0] = o[n][m][1] = o[n][m][2] = o[n][m][3] = 0.f;
        l[n][0] = l[n][1] = l[n][2] = l[n][3] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          base[n][e] = 0.f;
          sl[n][e] = c.factor[8 * n + 2 * tig + e];
          poison[n][e] = false;
        }
      }
      float limit = -INFINITY;   // weights above 2^limit move the base
      const int ta = 4 * (gid >> 1) + (gid & 1);   // of a half tile: this lane's first key
      int slot = 0;
      for (int k = k0 + warp; k < k1; k += kFewWarps) {
        wait_copies<X::kStages - 1>();
        __syncwarp();
        const int t0 = (first / kTile + k) * kTile;
        const uint32_t kt = ring + (uint32_t)(slot * X::kStage), vt = kt + X::kHalf;
        const bool edge = ((missing >> slot) & 1u) || t0 + (kTile - 1) > T - L ||
                          (a.window > 0 && (long long)t0 < (long long)T - a.window);
        // ---- S^T = K Q^T
        float s[2][kColumns][4];
#pragma unroll
        for (int n = 0; n < kColumns; ++n)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) s[hf][n][0] = s[hf][n][1] = s[hf][n][2] = s[hf][n][3] = 0.f;
        {
          constexpr int kW = kFour ? D / 32 : D / 16;   // words of a row a lane
          constexpr int kAt = kW < 4 ? kW : 4;          // of them at a time
          uint32_t sc[2][2];
          if constexpr (kFour) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              // bytes gid % 2 and + 2 of the quad's words: the lane's two keys
              const uint32_t at = kt + (uint32_t)(X::kCodes + (4 * hf + (gid >> 1)) * (D / 4) +
                                                  tig * (D / 16));
              const uint32_t sel = (gid & 1) ? 0x7351u : 0x6240u;
              uint2 w;
              if constexpr (D == 128) {
                w = lds8(at);
              } else {
                w.x = lds4(at);
                w.y = w.x;
              }
              e4m3x4_to_f16x2x2(prmt(w.x, w.y, sel), sc[hf][0], sc[hf][1]);
            }
          }
          constexpr int kPer = kFour ? 2 : 1;   // steps a word
#pragma unroll
          for (int w0 = 0; w0 < kW; w0 += kAt) {
            uint32_t kw[2][2][kAt];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int r = 16 * hf + ta + 2 * e;
                const uint32_t row = kt + (uint32_t)(r * X::kRowBytes);
                const int z = X::swizzle(r);
                if constexpr (kAt == 4) {
                  const uint4 u = lds16(row + (uint32_t)((((kW / 4) * tig + w0 / 4) ^ z) << 4));
                  kw[hf][e][0] = u.x; kw[hf][e][1] = u.y; kw[hf][e][2] = u.z; kw[hf][e][3] = u.w;
                } else {
                  const uint2 u = lds8(row + (uint32_t)((((tig >> 1) ^ z) << 4) + 8 * (tig & 1)));
                  kw[hf][e][0] = u.x; kw[hf][e][1] = u.y;
                }
              }
#pragma unroll
            for (int w = 0; w < kAt; ++w) {
              uint32_t f[2][2][2 * kPer];
#pragma unroll
              for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  if constexpr (kFour) {
                    uint32_t x[4];
                    e2m1x8_to_f16x2(kw[hf][e][w], x);
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                      f[hf][e][m] = w < 2 ? hmul2_lo(x[m], sc[hf][e]) : hmul2_hi(x[m], sc[hf][e]);
                  } else {
                    e4m3x4_to_f16x2x2(kw[hf][e][w], f[hf][e][0], f[hf][e][1]);
                  }
                }
#pragma unroll
              for (int u = 0; u < kPer; ++u)
#pragma unroll
                for (int n = 0; n < kColumns; ++n)
                  if (n < cols) {
                    const uint2 q = c.q[kPer * (w0 + w) + u][n][lane];
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
                      mma_16816<false>(s[hf][n], f[hf][0][2 * u], f[hf][1][2 * u],
                                       f[hf][0][2 * u + 1], f[hf][1][2 * u + 1], q.x, q.y);
                  }
            }
          }
        }
        // ---- weights 2^(s - base): the base is the largest score less kShift when it
        // is set and stays until a weight would pass 2^kTop
        uint32_t live[kColumns][2], nan = 0u;
        if (edge) {
          uint32_t there = kAll;
          if ((missing >> slot) & 1u)
#pragma unroll
            for (int b = 0; b < X::kStages; ++b)
              if (b == slot) there = ~bads[b];
#pragma unroll
          for (int n = 0; n < kColumns; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int p = c.pos[8 * n + 2 * tig + e];
              uint32_t m = p < t0 ? 0u : (p - t0 >= 31 ? kAll : (2u << (p - t0)) - 1u);
              const long long from = (long long)p - a.window + 1 - t0;
              if (a.window > 0 && from > 0) m = from > 31 ? 0u : m & (kAll << from);
              live[n][e] = m & there;
            }
        }
        float mx[kColumns][2], top = -INFINITY;
#pragma unroll
        for (int n = 0; n < kColumns; ++n)
          if (n < cols) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                s[hf][n][e] = fmaf(s[hf][n][e], sl[n][e & 1], -base[n][e & 1]);
                if (edge && !((live[n][e & 1] >> (16 * hf + ta + (e >> 1) * 2)) & 1u))
                  s[hf][n][e] = -INFINITY;
              }
#pragma unroll
            for (int e = 0; e < 2; ++e)
              mx[n][e] = fmaxf(max3f(s[0][n][e], s[0][n][2 + e], s[1][n][e]), s[1][n][2 + e]);
            top = max3f(top, mx[n][0], mx[n][1]);
          }
        if (__any_sync(kAll, top > limit)) {
          bool set = true;
#pragma unroll
          for (int n = 0; n < kColumns; ++n)
            if (n < cols) {
              float alpha[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float x = mx[n][e];
                x = fmaxf(x, __shfl_xor_sync(kAll, x, 4));
                x = fmaxf(x, __shfl_xor_sync(kAll, x, 8));
                x = fmaxf(x, __shfl_xor_sync(kAll, x, 16));
                // without weights so far the base goes anywhere, else only up
                const bool fresh = l[n][e] == 0.f;
                float d = x - kShift;
                if (x == -INFINITY || (!fresh && d < 0.f)) d = 0.f;
                set = set && (!fresh || x > -INFINITY);
                alpha[e] = fresh ? 1.f : ex2_approx(-d);
                base[n][e] += d;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                  s[hf][n][e] -= d;
                  s[hf][n][2 + e] -= d;
                }
                l[n][e] *= alpha[e];
              }
#pragma unroll
              for (int m = 0; m < D / 16; ++m) {
                o[n][m][0] *= alpha[0];
                o[n][m][1] *= alpha[1];
                o[n][m][2] *= alpha[0];
                o[n][m][3] *= alpha[1];
              }
            }
          limit = __all_sync(kAll, set) ? kTop : -INFINITY;
        }
        uint32_t pb[2][kColumns][2];
#pragma unroll
        for (int n = 0; n < kColumns; ++n)
          if (n < cols) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
              for (int r = 0; r < 2; ++r)
                pb[hf][n][r] = movmatrix_trans(
                    pack2<false>(ex2_approx(s[hf][n][2 * r]), ex2_approx(s[hf][n][2 * r + 1])));
              // their sums, by a row of ones: the weights as they are used
              constexpr uint32_t kOnes = 0x3c003c00u;
              mma_16816<false>(l[n], kOnes, kOnes, kOnes, kOnes, pb[hf][n][0], pb[hf][n][1]);
            }
          }
        // ---- O^T += V^T P^T: this lane's four keys of a half, its D / 8 elements
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          constexpr int kW = kFour ? D / 64 : D / 32;   // words of a row a lane
          uint32_t vw[4][kW], s01 = 0u, s23 = 0u;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = 16 * hf + 4 * tig + j;
            const uint32_t row = vt + (uint32_t)(r * X::kRowBytes);
            const int z = X::swizzle(r);
            if constexpr (kW == 4) {
              const uint4 u = lds16(row + (uint32_t)((gid ^ z) << 4));
              vw[j][0] = u.x; vw[j][1] = u.y; vw[j][2] = u.z; vw[j][3] = u.w;
            } else if constexpr (kW == 2) {
              const uint2 u = lds8(row + (uint32_t)((((gid >> 1) ^ z) << 4) + 8 * (gid & 1)));
              vw[j][0] = u.x; vw[j][1] = u.y;
            } else {
              vw[j][0] = lds4(row + (uint32_t)((((gid >> 2) ^ z) << 4) + 4 * (gid & 3)));
            }
          }
          uint32_t sc = 0u;
          if constexpr (kFour)
            sc = lds4(vt + (uint32_t)(X::kCodes + (4 * hf + tig) * (D / 4) +
                                      (D == 128 ? gid : gid >> 1) * 4));
          if (edge) {
            // rows of which nothing is loaded, or which nobody attends to, and NaN
            // become zeros: a weight of zero times NaN would reach other rows
            uint32_t any = 0u;
#pragma unroll
            for (int n = 0; n < kColumns; ++n)
              if (n < cols) any |= live[n][0] | live[n][1];
            any |= __shfl_xor_sync(kAll, any, 1);
            any |= __shfl_xor_sync(kAll, any, 2);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int t = 16 * hf + 4 * tig + j;
              const bool in = ((any >> t) & 1u) != 0u;
              uint32_t odd = kFour ? nan_bytes(sc) & (0x80u << (8 * j)) : 0u;
              if constexpr (!kFour)
#pragma unroll
                for (int w = 0; w < kW; ++w) odd |= nan_bytes(vw[j][w]);
              if (in && odd) nan |= 1u << t;
              if (!in || odd) {
                if constexpr (kFour) {
                  sc &= ~(0xffu << (8 * j));
                } else {
#pragma unroll
                  for (int w = 0; w < kW; ++w) vw[j][w] = 0u;
                }
              }
            }
          }
          if constexpr (kFour) e4m3x4_to_f16x2x2(sc, s01, s23);
#pragma unroll
          for (int w = 0; w < kW; ++w) {
            const uint32_t v0 = vw[0][w], v1 = vw[1][w], v2 = vw[2][w], v3 = vw[3][w];
            constexpr int kM = kFour ? 4 : 2;   // m-tiles a word
            uint32_t x[kM][4];
            if constexpr (kFour) {
              constexpr uint32_t kLow = 0x0f0f0f0fu;
              // bytes of two keys' codes of one head_dim: even and odd elements
              uint32_t a0[4], a1[4], a2[4], a3[4];
              e2m1x8_to_f16x2((v0 & kLow) | ((v1 << 4) & ~kLow), a0);
              e2m1x8_to_f16x2(((v0 >> 4) & kLow) | (v1 & ~kLow), a1);
              e2m1x8_to_f16x2((v2 & kLow) | ((v3 << 4) & ~kLow), a2);
              e2m1x8_to_f16x2(((v2 >> 4) & kLow) | (v3 & ~kLow), a3);
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                x[b][0] = hmul2(a0[b], s01);
                x[b][1] = hmul2(a1[b], s01);
                x[b][2] = hmul2(a2[b], s23);
                x[b][3] = hmul2(a3[b], s23);
              }
            } else {
              e4m3x4_to_f16x2x2(prmt(v0, v1, 0x5140u), x[0][0], x[0][1]);
              e4m3x4_to_f16x2x2(prmt(v2, v3, 0x5140u), x[0][2], x[0][3]);
              e4m3x4_to_f16x2x2(prmt(v0, v1, 0x7362u), x[1][0], x[1][1]);
              e4m3x4_to_f16x2x2(prmt(v2, v3, 0x7362u), x[1][2], x[1][3]);
            }
#pragma unroll
            for (int b = 0; b < kM; ++b)
#pragma unroll
              for (int n = 0; n < kColumns; ++n)
                if (n < cols)
                  mma_16816<false>(o[n][kM * w + b], x[b][0], x[b][1], x[b][2], x[b][3],
                                   pb[hf][n][0], pb[hf][n][1]);
          }
        }
        if (edge) {
          nan = __reduce_or_sync(kAll, nan);
          if (nan)
#pragma unroll
            for (int n = 0; n < kColumns; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) poison[n][e] = poison[n][e] || (live[n][e] & nan) != 0u;
        }
        __syncwarp();   // every lane has read the stage
        if (next < k1) issue(slot);
        commit_copies();
        if (++slot == X::kStages) slot = 0;
      }
      wait_copies<0>();
      __syncthreads();   // the rings are idle
      // ---- the warps' sums, joined: [warp][row][D]
      float* const sums = reinterpret_cast<float*>(c.data);
#pragma unroll
      for (int n = 0; n < kColumns; ++n)
        if (n < cols)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * n + 2 * tig + e;
            float4* const dst =
                reinterpret_cast<float4*>(sums + ((size_t)warp * kFewRows + r) * D + (D / 8) * gid);
#pragma unroll
            for (int m = 0; m < D / 16; m += 2)
              dst[m / 2] = make_float4(o[n][m][e], o[n][m][2 + e], o[n][m + 1][e], o[n][m + 1][2 + e]);
            if (gid == 0) {
              c.ml[warp][0][r] = l[n][e] == 0.f ? -INFINITY : base[n][e];
              c.ml[warp][1][r] = poison[n][e] ? __uint_as_float(0x7fffffffu) : l[n][e];
            }
          }
      __syncthreads();
      const bool whole = k0 == 0 && k1 == nt;
      float* const rec =
          a.few_rec + ((size_t)blockIdx.x * 2 + (k0 == 0 ? 1 : 0)) * few_rec_floats(D);
      constexpr int kVecs = D / 4;
      // a row with a NaN in it is NaN
      constexpr int kTurnsOut = (kFewRows * kVecs + kFewThreads - 1) / kFewThreads;
      float4 acc[kTurnsOut];
      float ms[kTurnsOut], ls[kTurnsOut];
#pragma unroll
      for (int u = 0; u < kTurnsOut; ++u) {
        const int v = tid + u * kFewThreads, r = v / kVecs, col = 4 * (v % kVecs);
        if (r >= rows) break;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) m = fmaxf(m, c.ml[w][0][r]);
        const float from = m == -INFINITY ? 0.f : m;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
          const float f = ex2_approx(c.ml[w][0][r] - from);
          const float4 x = *reinterpret_cast<const float4*>(sums + ((size_t)w * kFewRows + r) * D + col);
          sum = fmaf(c.ml[w][1][r], f, sum);
          y.x = fmaf(x.x, f, y.x);
          y.y = fmaf(x.y, f, y.y);
          y.z = fmaf(x.z, f, y.z);
          y.w = fmaf(x.w, f, y.w);
        }
        const float all = (y.x + y.y) + (y.z + y.w);
        if (all != all) c.bad[r] = 1;   // (sums of finite values do not overflow here)
        acc[u] = y;
        ms[u] = m;
        ls[u] = sum;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kTurnsOut; ++u) {
        const int v = tid + u * kFewThreads, r = v / kVecs, col = 4 * (v % kVecs);
        if (r >= rows) break;
        if (c.bad[r]) ls[u] = __uint_as_float(0x7fffffffu);
        if (whole) {
          const float mul = ls[u] == 0.f ? 0.f : a.v_scale / ls[u];
          const int tok = r / a.G;
          *reinterpret_cast<uint2*>(a.out + ((size_t)(q0 + tok) * a.Hq + (size_t)h * a.G +
                                             (r - tok * a.G)) * D + col) =
              make_uint2(pack2<kBF16>(acc[u].x * mul, acc[u].y * mul),
                         pack2<kBF16>(acc[u].z * mul, acc[u].w * mul));
        } else {
          *reinterpret_cast<float4*>(rec + (size_t)r * D + col) = acc[u];
          if (col == 0) {
            rec[(size_t)kFewRows * D + r] = ms[u];
            rec[(size_t)kFewRows * (D + 1) + r] = ls[u];
          }
        }
      }
      __syncthreads();
      if (!whole) {
        // ---- a context cut between blocks: the blocks that hold tiles of it
        if (warp == 0) {
          int f = blockIdx.x, e = blockIdx.x;
          while (f > 0 && c.bound[f] > i0) --f;
          while (e + 1 < nb && c.bound[e + 1] < i0 + nt + kStartTiles) ++e;
          int n = 0, end = f;
          for (int b0 = f; b0 <= e; b0 += 32) {
            const int b = b0 + lane;
            bool in = false, begins = false;
            if (b <= e) {
              const int s0 = tile_at(c.bound[b]);
              in = s0 < tile_at(c.bound[b + 1]);
              begins = s0 == 0;
            }
            const uint32_t all = __ballot_sync(kAll, in);
            if (in)
              c.parts[n + __popc(all & ((1u << lane) - 1u))] = (uint16_t)(b * 2 + (begins ? 1 : 0));
            n += __popc(all);
            if (all) end = b0 + 31 - __clz(all);
          }
          if (lane == 0) {
            c.nparts = n;
            // releases this block's record (ordered before by the barrier), acquires
            // those counted before it
            uint32_t* const cnt = a.few_count + end;
            const bool done = atom_add_acq_rel_gpu(cnt, 1u) + 1u == (uint32_t)n;
            if (done) *cnt = 0u;   // ready for the next call
            c.last = done ? 1 : 0;
          }
        }
        __syncthreads();
        if (c.last) {   // the last record: join them all, in the order of the keys
          const int n = c.nparts;
          if (tid < rows) {
            float m = -INFINITY, ls = 0.f;
            for (int k = 0; k < n; ++k) {
              const float* const p = a.few_rec + (size_t)c.parts[k] * few_rec_floats(D) +
                                     (size_t)kFewRows * D + tid;
              const float pm = __ldcg(p), pl = __ldcg(p + kFewRows);
              const float mn = fmaxf(m, pm), from = mn == -INFINITY ? 0.f : mn;
              ls = ls * ex2_approx(m - from) + pl * ex2_approx(pm - from);
              m = mn;
            }
            c.join[tid][0] = m == -INFINITY ? 0.f : m;
            c.join[tid][1] = ls == 0.f ? 0.f : a.v_scale / ls;
          }
          __syncthreads();
          for (int v = tid; v < rows * kVecs; v += kFewThreads) {
            const int r = v / kVecs, col = 4 * (v % kVecs);
            const float m = c.join[r][0], mul = c.join[r][1];
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < n; k += 4) {
              float4 x[4];
              float w[4];
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                const float* const p =
                    a.few_rec + (size_t)c.parts[min(k + b, n - 1)] * few_rec_floats(D);
                x[b] = __ldcg(reinterpret_cast<const float4*>(p + (size_t)r * D + col));
                w[b] = __ldcg(p + (size_t)kFewRows * D + r);
              }
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                const float f = k + b < n ? ex2_approx(w[b] - m) : 0.f;
                acc.x = fmaf(x[b].x, f, acc.x);
                acc.y = fmaf(x[b].y, f, acc.y);
                acc.z = fmaf(x[b].z, f, acc.z);
                acc.w = fmaf(x[b].w, f, acc.w);
              }
            }
            const int tok = r / a.G;
            *reinterpret_cast<uint2*>(a.out + ((size_t)(q0 + tok) * a.Hq + (size_t)h * a.G +
                                               (r - tok * a.G)) * D + col) =
                make_uint2(pack2<kBF16>(acc.x * mul, acc.y * mul),
                           pack2<kBF16>(acc.z * mul, acc.w * mul));
          }
          __syncthreads();
        }
      }
    } else {
      walk_on();
      __syncthreads();
    }
    turn ^= 1;
    take();
  }
}

}  // namespace

}  // namespace pa
