// Multi-query paged attention over quantized KV caches (E4M3 and 4-bit pools):
// chunks of new tokens, single tokens among them, causal, with an optional
// sliding window.
//
// What it computes, with K and V the values the codes stand for before the
// tensor's scale, for the new token at position p of its sequence:
//   s_t = scale * k_scale * q . K_t,  o = v_scale * sum_t softmax(s)_t V_t,
// t over [max(0, p - window + 1), p].
//
// A row is one query head of one new token; a tile is the 128 rows of 128 / G
// tokens of one KV head, a pair two consecutive tiles A and B, which share the
// stream of keys.  Codes are exact in binary16 (an E4M3 value has 4 significant
// bits, E2M1 times its scale 6), so the products run on the fifth-generation
// tensor cores in binary16 with fp32 sums in tensor memory.
//
// Roles of a block of 16 warps, one block an SM:
//  * warps 8-11 (loaders) walk the block's share of the work.  A thread copies
//    4 rows x 16 elements of K and of V of a stage of 64 keys to shared memory
//    as they lie in the pool (asynchronous copies into a ring that only the
//    copying thread reads, so no barrier), converts them some stages later, and
//    stores them as 16-bit operands with the 128-byte swizzle.  At a part's
//    start they bring its query rows in, as binary16.
//  * warps 12 and 13 (one thread each, a tile each): S = Q K^T of a stage.
//  * warps 0-3 (tile A) and 4-7 (tile B): thread r owns row r, tensor memory
//    lane r.  It reads its scores, masks them, writes P = 2^(s - m) and keeps
//    the row's sum; m moves only when a weight would pass 2^kTop, and then the
//    row of O is rescaled in tensor memory.
//  * warp 14 (one thread, both tiles): O += P V, P from tensor memory.
// A pair without a second tile gives its stages to the tiles in turn: both hold
// the same rows and end with partial results, which tile A's warps join.
//
// The split.  The pairs of all sequences and KV heads, in that order, are a line
// on which a pair is kStart + (its attended tokens) long; it is cut into equal
// shares, one a block.  A pair cut between blocks leaves one record (O, m, l) a
// tile and block in the workspace, and the last block to count its record joins
// them, always in the order of the keys: no block waits for another, and the
// result depends on nobody's speed.
#pragma once

#include <cmath>
#include <mutex>

#include "pa_fp4.cuh"
#include "pa_host.h"

namespace pa {

namespace {

constexpr int kKeys = 64;                 // of a stage
constexpr int kLoaders = 8;               // first loader warp
constexpr int kScore = 12;                // warps 12 and 13
constexpr int kPv = 14;
constexpr int kAlloc = 15;
constexpr int kThreads = 512;
constexpr int kMaxGrid = 256;
// A pair's start and end cost what this many tokens do.
constexpr int kStart = 128;
// Small batches take a block for every kLeast of the line.
constexpr int kLeast = 384;
// The exponentials' reference is a maximum less kShift when it is set and stays
// until a weight would pass 2^kTop: binary16 holds weights down to 2^-14 - kShift
// of the maximum with all their bits.
constexpr float kShift = 7.f, kTop = 15.f, kTopPow = 32768.f;
// Registers of the roles: softmax, loaders, the others (sum 4 x 128 a thread).
constexpr int kRegsSoftmax = 168, kRegsLoad = 120, kRegsOther = 56;
static_assert(2 * kRegsSoftmax + kRegsLoad + kRegsOther == 4 * 128, "the launch's registers");

struct Args {
  const uint16_t* q;
  uint16_t* out;
  const uint8_t* kc;
  const uint8_t* vc;
  const int32_t* bt;
  const int32_t* seq_lens;
  const int32_t* query_start;
  uint32_t* ws_count;       // [grid][2], zero between calls
  float* ws_rec;            // [grid][2][2] records of rec_floats(D)
  int32_t* err;
  long long num_blocks, total_q;
  int num_seqs, stride, Hq, H, G, BM, log2B, window;
  float scale_log2, v_scale;
};

constexpr int kTileRows = 128;
// o[128][D], m[128], l[128]
__host__ __device__ constexpr size_t rec_floats(int D) { return (size_t)kTileRows * (D + 2); }

// A stage as it lies in the pool: units of 4 rows x 16 elements, kPiece bytes a
// row, and for 4-bit pools the unit's four scales.
template <int D, bool kFour>
struct Raw {
  static constexpr int kGroups = D / 16;
  static constexpr int kUnits = (kKeys / 4) * kGroups;
  static constexpr int kPiece = kFour ? 8 : 16;
  static constexpr int kHalf = 4 * kUnits * kPiece + (kFour ? 4 * kUnits : 0);   // K, then V
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kRing = D == 64 ? 6 : (kFour ? 5 : 3);   // stages in flight
};

template <int D>
struct Tiles {
  static constexpr int kStages = D == 64 ? 6 : 3;
  static constexpr int kPlanes = D / 64;
  static constexpr uint32_t kPart = kKeys * D * 2;          // K or V of a stage
  static constexpr uint32_t kStage = 2 * kPart;
  static constexpr uint32_t kPlane = kKeys * 128;           // 64 columns of it
  static constexpr uint32_t kQPlane = kTileRows * 128;
  static constexpr uint32_t kQTile = kPlanes * kQPlane;
};

// flags of a stage
enum : int {
  kStop = 1, kFirst = 2, kLast = 4, kActA = 8, kActB = 16, kFirstA = 32, kFirstB = 64,
  kLastA = 128, kLastB = 256, kAlt = 512, kWholeA = 1024, kWholeB = 2048, kBegins = 4096,
  kHasB = 8192
};

// What the loaders say about a stage, beside its keys.
struct Tag {
  int flags, kt, h, q0;             // q0: tile A's first q row
  int ntok_a, ntok_b, p0, lo;       // tokens, tile A's first position, first attended token
  int nkt_a, nkt, pad0, pad1;       // stages end of tile A, of the pair
  long long i0, len;                // the pair's place on the line, its length there
  uint32_t mask[4];                 // bits of keys: left out (2 words), NaN value rows (2 words)
};

template <int S>
struct Control {
  unsigned long long full[S], empty[S], seen[S];
  unsigned long long qempty, bdone, done[3];
  unsigned long long tile[2][8];    // s full, s free, p full[2], p empty[2], o free
  alignas(16) Tag tag[S];
  float factor[S][2][kTileRows];    // of a part's rows: what scores are multiplied by
  float ml[kTileRows][2];           // tile B's m and l, of a pair in turn
  volatile uint32_t pvq[2][8];      // records of products to issue: ring[4], tail, head, fin
  long long run_pref[kThreads];     // the line before each thread's run of sequences
  long long warp_tot[kThreads / 32];
  long long bound[kMaxGrid + 1];
  uint16_t parts[2][kMaxGrid];      // of a cut tile: its records
  int nparts[2];
  int last[2];
  uint32_t tmem;
  volatile int abort;
};
// places in Control::tile
enum : int { kSFull = 0, kSFree = 1, kPFull = 2, kPEmpty = 4, kOFree = 6 };

template <int D, bool kFour>
constexpr size_t smem_bytes() {
  return 1024 + Tiles<D>::kStages * Tiles<D>::kStage + 2 * Tiles<D>::kQTile +
         Raw<D, kFour>::kRing * Raw<D, kFour>::kStage + sizeof(Control<Tiles<D>::kStages>);
}

// D[tmem] (+)= A . B with A in tensor memory (M rows in lanes, K along columns,
// two 16-bit elements to one), B from shared memory
__device__ __forceinline__ void umma_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                            uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u));
}

// kBytes from global to shared memory; `on` false fills with zeros instead
template <int kBytes>
__device__ __forceinline__ void copy_piece(uint32_t dst, const uint8_t* src, bool on) {
  const int n = on ? kBytes : 0;
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src),
                 "n"(kBytes), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void commit_copies() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kPending>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr));
  return r;
}
__device__ __forceinline__ uint2 lds8(uint32_t addr) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr));
  return r;
}
__device__ __forceinline__ uint32_t lds4(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                      uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
// the 128 threads of a warpgroup
__device__ __forceinline__ void group_sync(int id) {
  asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}
// bytes of E4M3 codes that are NaN: 0x80 in their place
__device__ __forceinline__ uint32_t nan_bytes(uint32_t x) {
  return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Sequence i: its rows of q and its length; false (no tokens then) where they
// contradict each other or the table.
__device__ __forceinline__ bool load_seq(const Args& a, int i, int& q0, int& L, int& T) {
  const int s0 = __ldg(a.query_start + i), s1 = __ldg(a.query_start + i + 1);
  T = __ldg(a.seq_lens + i);
  const long long n = (long long)s1 - s0;
  const bool ok = s0 >= 0 && n >= 0 && s1 <= a.total_q && T >= 0 &&
                  (long long)T <= ((long long)a.stride << a.log2B) && n <= T;
  q0 = s0;
  L = ok ? (int)n : 0;
  return ok;
}

__device__ __forceinline__ int pairs_of(int L, const Args& a) {
  return (int)(((long long)L + 2 * a.BM - 1) / (2 * a.BM));
}

// The line's length of pairs 0 .. pr - 1 of a sequence with P of them (one KV
// head): pair j ends with token T - L + min(2 BM (j + 1), L) and begins with the
// first token its first row attends to.
__device__ __forceinline__ long long line_before(long long pr, long long P, int L, int T,
                                                 const Args& a) {
  const long long base = (long long)T - L, w = 2 * a.BM;
  long long sum = kStart * pr;
  if (pr < P) sum += pr * base + w * (pr * (pr + 1) / 2);
  else if (P > 0) sum += (P - 1) * base + w * ((P - 1) * P / 2) + T;
  if (a.window > 0) {   // less the sum of max(0, base + w j - window + 1)
    const long long x = (long long)a.window - 1 - base;
    const long long j0 = x < 0 ? 0 : x / w + 1;
    if (pr > j0) sum -= w * (pr * (pr - 1) / 2 - j0 * (j0 - 1) / 2) - x * (pr - j0);
  }
  return sum;
}

// The first stage of a pair that begins at or behind `at` on the line, counted
// from the pair's place (stages are 64 keys on from token 0; a pair's first one
// stands at kStart).
__device__ __forceinline__ int stage_at(long long at, int lo, int nkt) {
  const long long r = at - kStart;
  if (r <= 0) return lo / kKeys;
  const long long k = (lo + r + kKeys - 1) / kKeys;
  return k < nkt ? (int)k : nkt;
}

// A place in a block's share of the line.
struct Walk {
  int i, q0, L, T, P;          // sequence
  int h, pr, lo, end;          // pair: first attended token, end of the attended ones
  int k, k0, k1;               // stage; the stages of this block's part of the pair
  long long i0, u0, u1;        // the pair's place; the block's share
  bool done;

  __device__ __forceinline__ long long length() const { return (long long)kStart + end - lo; }
  __device__ __forceinline__ int nkt() const { return (end - 1) / kKeys + 1; }

  // from the pair on to the next stage there is
  __device__ __forceinline__ void settle(const Args& a) {
    while (true) {
      if (i >= a.num_seqs || i0 >= u1) {
        done = true;
        return;
      }
      const long long w = 2 * a.BM, base = (long long)T - L;
      end = (int)(base + min(w * (pr + 1), (long long)L));
      const long long first = base + w * pr - a.window + 1;
      lo = a.window > 0 && first > 0 ? (int)first : 0;
      k0 = stage_at(u0 - i0, lo, nkt());
      k1 = stage_at(u1 - i0, lo, nkt());
      k = k0;
      if (k0 < k1) return;
      next_pair(a);
    }
  }
  __device__ __forceinline__ void next_pair(const Args& a) {
    i0 += length();
    if (++pr < P) return;
    pr = 0;
    if (++h < a.H) return;
    h = 0;
    P = 0;
    while (P == 0 && ++i < a.num_seqs) {
      load_seq(a, i, q0, L, T);
      P = pairs_of(L, a);
    }
  }
  __device__ __forceinline__ void advance(const Args& a) {
    if (++k < k1) return;
    next_pair(a);
    settle(a);
  }
  // to place u0 of the line
  __device__ __forceinline__ void start(const Args& a, const long long* run_pref, int per,
                                        long long from, long long to) {
    u0 = from;
    u1 = to;
    done = false;
    int r = 0;   // the last run that starts at or before u0
#pragma unroll
    for (int b = kThreads / 2; b > 0; b >>= 1)
      if (r + b < kThreads && run_pref[r + b] <= u0) r += b;
    long long rem = u0 - run_pref[r], one = 0;
    i = r * per;
    while (i < a.num_seqs) {
      load_seq(a, i, q0, L, T);
      P = pairs_of(L, a);
      one = line_before(P, P, L, T, a);
      if (rem < one * a.H) break;
      rem -= one * a.H;
      ++i;
    }
    if (i >= a.num_seqs) {   // lengths that changed during the call
      done = true;
      return;
    }
    h = (int)(rem / one);
    rem -= one * h;
    int below = 0, above = P;   // the last pair that starts at or before the place
    while (above - below > 1) {
      const int mid = (below + above) >> 1;
      if (line_before(mid, P, L, T, a) <= rem) below = mid;
      else above = mid;
    }
    pr = below;
    i0 = u0 - (rem - line_before(pr, P, L, T, a));
    settle(a);
  }
};

template <int D, bool kBF16, bool kFour>
__global__ void __launch_bounds__(kThreads, 1) prefill_quant_kernel(const Args a) {
  using R = Raw<D, kFour>;
  using X = Tiles<D>;
  constexpr int S = X::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw0 = smem_u32(smem_raw);
  const uint32_t stages = (raw0 + 1023u) & ~1023u;
  const uint32_t qtiles = stages + S * X::kStage;
  const uint32_t ring = qtiles + 2 * X::kQTile;
  Control<S>& c = *reinterpret_cast<Control<S>*>(smem_raw + (ring - raw0) + R::kRing * R::kStage);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&c.full[s]), 128);      // the loaders' threads
      mbar_init(smem_u32(&c.empty[s]), 4);       // per tile: a K share, a V share
      mbar_init(smem_u32(&c.seen[s]), 8);        // a softmax warp each
    }
    mbar_init(smem_u32(&c.qempty), 2);           // a commit of each score issuer
    mbar_init(smem_u32(&c.bdone), 128);          // tile B's threads
    for (int k = 0; k < 3; ++k) mbar_init(smem_u32(&c.done[k]), 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&c.tile[t][kSFull]), 1);
      mbar_init(smem_u32(&c.tile[t][kSFree]), 128);
      for (int p = 0; p < 2; ++p) {
        mbar_init(smem_u32(&c.tile[t][kPFull + p]), 128);
        mbar_init(smem_u32(&c.tile[t][kPEmpty + p]), 1);
      }
      mbar_init(smem_u32(&c.tile[t][kOFree]), 128);
      for (int w = 0; w < 8; ++w) c.pvq[t][w] = 0u;
    }
    c.abort = 0;
    fence_barrier_init();
  }
  grid_dep_wait();

  // ---- the line: every thread sums a run of sequences ----------------------
  const int per = (a.num_seqs + kThreads - 1) / kThreads;
  const int run0 = min(a.num_seqs, tid * per), run1 = min(a.num_seqs, run0 + per);
  long long mine = 0;
  bool odd = false;
  for (int i = run0; i < run1; ++i) {
    int q0, L, T;
    odd |= !load_seq(a, i, q0, L, T);
    const int P = pairs_of(L, a);
    mine += line_before(P, P, L, T, a) * a.H;
  }
  long long incl = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long n = __shfl_up_sync(0xffffffffu, incl, s);
    if (lane >= s) incl += n;
  }
  if (lane == 31) c.warp_tot[warp] = incl;
  odd = __syncthreads_or(odd) != 0;
  long long off = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) off += c.warp_tot[w];
    total += c.warp_tot[w];
  }
  c.run_pref[tid] = off + incl - mine;
  if (tid == 0) grid_dep_launch();
  if (odd) {   // sequences that contradict themselves: reported, their rows cleared
    for (int i = blockIdx.x; i < a.num_seqs; i += gridDim.x) {
      int q0, L, T;
      if (load_seq(a, i, q0, L, T)) continue;
      if (tid == 0) set_error(a.err, PA_DEVERR_SEQ_LEN);
      const long long r0 = max(q0, 0);
      const long long r1 = min((long long)__ldg(a.query_start + i + 1), a.total_q);
      uint4* dst = reinterpret_cast<uint4*>(a.out + (size_t)r0 * a.Hq * D);
      for (long long e = tid; e < (r1 - r0) * a.Hq * (D / 8); e += kThreads)
        dst[e] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  const long long nb = min((long long)gridDim.x, (total + kLeast - 1) / kLeast);
  if ((long long)blockIdx.x >= nb) return;
  if (tid <= nb) c.bound[tid] = total * tid / nb;
  if (warp == kAlloc) {
    tmem_alloc(smem_u32(&c.tmem), 512);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;

  // a wait whose outcome is the same in every lane of the warp
  auto wait_warp = [&](unsigned long long& bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar), parity,
                                                     const_cast<volatile int*>(&c.abort))) != 0;
  };
  auto give_up = [&]() {   // by one thread: the other roles leave on the flag
    if (!c.abort) set_error(a.err, PA_DEVERR_TIMEOUT);
    c.abort = 1;
  };

  if (warp >= kScore) {
    setmaxnreg_dec<kRegsOther>();
    if (warp < kPv && lane == 0) {
      // ===================== score products of tile t =====================
      // The next stage's S = Q K^T as soon as its keys are there, the S buffer
      // and the P region its weights will go to are free, and at most one of
      // the tile's O += P V is still to be issued (the tensor pipe executes in
      // issue order).  Every product leaves a record for the O issuer: the
      // stage's slot (bits 0-2), a part's first (3), wait for O (4) with
      // parity (5).
      static_assert(S <= 8, "slots take 3 bits");
      const int t = warp - kScore;
      const int act = t == 0 ? kActA : kActB, first = t == 0 ? kFirstA : kFirstB;
      constexpr uint32_t id_s = umma_idesc_f16(false, kTileRows, kKeys, false);
      volatile uint32_t* const q = c.pvq[t];
      unsigned long long* const tb = c.tile[t];
      const uint32_t tcol = tmem + (uint32_t)(256 * t);
      const uint64_t dq[2] = {umma_desc_sw128(qtiles, 16, 1024),
                              umma_desc_sw128(qtiles + (uint32_t)t * X::kQTile, 16, 1024)};
      int rt = 0, ni = 0, st = 0;   // records pushed (scores issued), parts started, slot
      uint32_t ph = 0u;
      bool ok = true;
      long long t_last = clock64();
      while (true) {
        bool progressed = false;
        if (rt - (int)q[5] < 2 && mbar_test(smem_u32(&c.full[st]), ph)) {
          const int flags = *const_cast<volatile int*>(&c.tag[st].flags);
          if (flags & kStop) break;
          bool ready = true;
          if (flags & act) {
            if (rt >= 1) ready = mbar_test(smem_u32(&tb[kSFree]), (uint32_t)(rt - 1) & 1u);
            if (ready && rt >= 2)
              ready = mbar_test(smem_u32(&tb[kPEmpty + (rt & 1)]), (uint32_t)((rt >> 1) - 1) & 1u);
            if (ready) {
              tc_fence_after();
              const uint64_t da = dq[(flags & kAlt) ? 0 : 1];
              const uint64_t db = umma_desc_sw128(stages + (uint32_t)st * X::kStage, 16, 1024);
              // K steps of 16 columns: 32 bytes on within a 64-column plane
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t o = (uint32_t)(ks & 3) * 32u, p = (uint32_t)(ks >> 2);
                umma_f16(tcol, da + ((p * X::kQPlane + o) >> 4), db + ((p * X::kPlane + o) >> 4),
                         id_s, ks > 0);
              }
              umma_commit(smem_u32(&tb[kSFull]));
              umma_commit(smem_u32(&c.empty[st]));   // the K share
              uint32_t rc = (uint32_t)st;
              if (flags & first) {
                rc |= 8u;
                if (ni > 0) rc |= 16u | ((uint32_t)((ni - 1) & 1) << 5);
                ++ni;
              }
              q[rt & 3] = rc;
              __threadfence_block();   // the record before the tail that publishes it
              q[4] = (uint32_t)(++rt);
            }
          } else {   // not this tile's: both shares
            umma_commit(smem_u32(&c.empty[st]));
            mbar_arrive(smem_u32(&c.empty[st]));
          }
          if (ready) {
            if (flags & kLast) umma_commit(smem_u32(&c.qempty));   // the queries are read
            if (++st == S) {
              st = 0;
              ph ^= 1u;
            }
            progressed = true;
          }
        }
        if (progressed) {
          t_last = clock64();
        } else {
          if (c.abort || clock64() - t_last > kWaitLimitCycles) {
            ok = false;
            break;
          }
          __nanosleep(20);   // the issue slots are the softmax warps'
        }
      }
      if (!ok) give_up();
      __threadfence_block();
      q[6] = 1u;   // no more records
      umma_commit(smem_u32(&c.done[t]));
      mbar_wait_bounded(smem_u32(&c.done[t]), 0u, nullptr);
    } else if (warp == kPv && lane == 0) {
      // ===================== O += P V of both tiles =====================
      constexpr uint32_t id_o = umma_idesc_f16(false, kTileRows, D, true);
      int rh[2] = {0, 0};   // records issued
      bool ok = true;
      long long t_last = clock64();
      auto try_pv = [&](int t, int& n) -> bool {
        volatile uint32_t* const q = c.pvq[t];
        if ((int)q[4] == n) return false;
        __threadfence_block();
        const uint32_t rc = q[n & 3];
        unsigned long long* const tb = c.tile[t];
        if (!mbar_test(smem_u32(&tb[kPFull + (n & 1)]), (uint32_t)(n >> 1) & 1u)) return false;
        if ((rc & 16u) && !mbar_test(smem_u32(&tb[kOFree]), (rc >> 5) & 1u)) return false;
        tc_fence_after();
        const int st = (int)(rc & 7u);
        const bool first = (rc & 8u) != 0u;
        const uint32_t tcol = tmem + (uint32_t)(256 * t);
        // V (64 keys x D) MN-major: 64-column planes kPlane apart, groups of 8
        // keys 1024 bytes apart; 16 keys a step, 8 columns of P
        const uint64_t dv = umma_desc_sw128(stages + (uint32_t)st * X::kStage + X::kPart,
                                            X::kPlane, 1024);
        const uint32_t p = tcol + 64u + 32u * (uint32_t)(n & 1);
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          umma_tmem_a(tcol + 128u, p + 8u * k, dv + ((uint32_t)k * 2048u >> 4), id_o,
                      !first || k > 0);
        umma_commit(smem_u32(&tb[kPEmpty + (n & 1)]));
        umma_commit(smem_u32(&c.empty[st]));   // the V share
        q[5] = (uint32_t)(++n);
        return true;
      };
      while (true) {
        bool progressed = try_pv(0, rh[0]);
        progressed = try_pv(1, rh[1]) || progressed;
        if (progressed) {
          t_last = clock64();
          continue;
        }
        if (c.pvq[0][6] && c.pvq[1][6]) {
          __threadfence_block();
          if ((int)c.pvq[0][4] == rh[0] && (int)c.pvq[1][4] == rh[1]) break;
        }
        if (c.abort || clock64() - t_last > kWaitLimitCycles) {
          ok = false;
          break;
        }
        __nanosleep(20);
      }
      if (!ok) give_up();
      umma_commit(smem_u32(&c.done[2]));
      mbar_wait_bounded(smem_u32(&c.done[2]), 0u, nullptr);
    }
    __syncwarp();
  } else if (warp >= kLoaders) {
    setmaxnreg_dec<kRegsLoad>();
    // ========================= loaders =========================
    const int x = tid - 32 * kLoaders;              // 0 .. 127
    const int u = x % R::kUnits, part0 = D == 64 ? x / R::kUnits : 0;
    constexpr int kParts = D == 64 ? 1 : 2;         // of K and V, a thread's
    const int ua = u / R::kGroups, g = u % R::kGroups;
    const int B = 1 << a.log2B;
    const int tok_r = x / a.G, head_r = x % a.G;    // of this thread's query row
    Walk cv;
    cv.start(a, c.run_pref, per, c.bound[blockIdx.x], c.bound[blockIdx.x + 1]);
    Walk ld = cv;
    // the block of this thread's unit of a stage; -2: none of its tokens is
    // attended to
    auto entry = [&](const Walk& w) -> int {
      if (w.done) return -2;
      const int t = w.k * kKeys + 4 * ua;
      if (t + 3 < w.lo || t >= w.end) return -2;
      return __ldg(a.bt + (size_t)w.i * a.stride + (t >> a.log2B));
    };
    uint32_t bads = 0;   // a bit per ring slot: the unit's block is out of range
    auto issue = [&](int slot, int ent) {
      const int t = ld.k * kKeys + 4 * ua;
      bool on = ent != -2;
      bads &= ~(1u << slot);
      if (on && (ent < 0 || (long long)ent >= a.num_blocks)) {
        set_error(a.err, PA_DEVERR_BLOCK_ID);
        bads |= 1u << slot;
        on = false;
      }
      const int e = on ? ent : 0, r = t & (B - 1);
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        const int kv = part0 + p;
        const uint8_t* const pool = kv ? a.vc : a.kc;
        const uint32_t dst = ring + (uint32_t)(slot * R::kStage + kv * R::kHalf + u * R::kPiece);
        if constexpr (kFour) {
          const uint8_t* const plane =
              pool + fp4_plane(e, a.H, on ? ld.h : 0, B * fp4_row_bytes(D));
          const uint8_t* const src = on ? plane + r * (D / 2) + 8 * g : pool;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            copy_piece<8>(dst + i * (R::kUnits * 8), on ? src + i * (D / 2) : pool,
                          on && t + i < ld.end);
          copy_piece<4>(ring + (uint32_t)(slot * R::kStage + kv * R::kHalf + 32 * R::kUnits + 4 * u),
                        on ? plane + fp4_scale_off<D>(B, r, g) : pool, on);
        } else {
          const size_t row = (size_t)a.H * D;
          const uint8_t* const src =
              on ? pool + ((size_t)e * B + r) * row + (size_t)ld.h * D + 16 * g : pool;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            copy_piece<16>(dst + i * (R::kUnits * 16), on ? src + i * row : pool,
                           on && t + i < ld.end);
        }
      }
      ld.advance(a);
    };
    {
      int ents[R::kRing];
      Walk w = cv;
#pragma unroll
      for (int n = 0; n < R::kRing; ++n) {
        ents[n] = entry(w);
        if (!w.done) w.advance(a);
      }
#pragma unroll
      for (int n = 0; n < R::kRing; ++n) {
        if (!ld.done) issue(n, ents[n]);
        commit_copies();   // a group a stage, issued or not
      }
    }
    int ent = entry(ld);
    int st = 0, slot = 0, parts = 0;
    uint32_t ph = 0u;
    bool ok = true;
    while (!cv.done) {
      ok = wait_warp(c.empty[st], ph ^ 1u) && wait_warp(c.seen[st], ph ^ 1u);
      const bool first = cv.k == cv.k0;
      const long long w2 = 2 * a.BM;
      const int left = (int)min((long long)cv.L - w2 * cv.pr, w2);   // the pair's tokens
      const int ntok_a = min(left, a.BM), ntok_b = left - ntok_a;
      const int q0 = cv.q0 + (int)(w2 * cv.pr);
      if (ok && first) {
        ok = wait_warp(c.qempty, ((uint32_t)parts & 1u) ^ 1u);
        ++parts;
        if (ok) {
          // ---- query rows: thread x row x of a tile, as binary16.  A bfloat16
          // row is brought into binary16's range by a power of two (its largest
          // magnitude into [1, 2)), which its score factor takes back; elements
          // 2^-14 below the largest lose bits below 2^-24 of it.
#pragma unroll 1
          for (int t = 0; t < (ntok_b > 0 ? 2 : 1); ++t) {
            const bool valid = x < a.BM * a.G && tok_r < (t ? ntok_b : ntok_a);
            uint32_t w[D / 2];
            const uint4* src = reinterpret_cast<const uint4*>(
                a.q + ((size_t)(valid ? q0 + t * a.BM + tok_r : 0) * a.Hq +
                       (valid ? cv.h * a.G + head_r : 0)) * D);
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
              const uint4 y = valid ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
              w[4 * j] = y.x; w[4 * j + 1] = y.y; w[4 * j + 2] = y.z; w[4 * j + 3] = y.w;
            }
            float back = 1.f;
            if constexpr (kBF16) {
              float mx = 0.f;
#pragma unroll
              for (int j = 0; j < D / 2; ++j) {
                const float2 f = unpack2<true>(w[j]);
                mx = max3f(mx, fabsf(f.x), fabsf(f.y));
              }
              // 2^e <= mx < 2^(e+1); zero, subnormal or infinite maxima keep a
              // factor whose inverse is a normal number
              const int e = min(max((int)(__float_as_uint(mx) >> 23), 1), 253);
              back = __uint_as_float((uint32_t)e << 23);
              const float to = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
              for (int j = 0; j < D / 2; ++j) {
                const float2 f = unpack2<true>(w[j]);
                w[j] = pack2<false>(f.x * to, f.y * to);
              }
            }
            const uint32_t dst = qtiles + (uint32_t)t * X::kQTile + (uint32_t)x * 128u;
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
              sts16(dst + (uint32_t)(j >> 3) * X::kQPlane + (uint32_t)((j ^ x) & 7) * 16u,
                    w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            c.factor[st][t][x] = a.scale_log2 * back;
          }
        }
      }
      if (!ok) {
        if (lane == 0) give_up();
        break;
      }
      // ---- the stage's keys and values to 16 bits
      wait_copies<R::kRing - 1>();
      const int t0 = cv.k * kKeys + 4 * ua;
      uint32_t nan = 0u;   // a bit per row of the unit
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        const int kv = part0 + p;
        const uint32_t src = ring + (uint32_t)(slot * R::kStage + kv * R::kHalf + u * R::kPiece);
        // row r of the unit: chunks 2 g and 2 g + 1 of its 128-byte plane rows.
        // Lanes of the other plane, or of the next unit of a 64-element row,
        // store them the other way round: no two lanes of eight share a bank.
        const uint32_t dst = stages + (uint32_t)st * X::kStage + (uint32_t)kv * X::kPart +
                             (uint32_t)(g >> 2) * X::kPlane + (uint32_t)(4 * ua) * 128u;
        const uint32_t turn = D == 128 ? (uint32_t)(g >> 2) : (uint32_t)(ua & 1);
        uint32_t s01 = 0u, s23 = 0u;
        if constexpr (kFour) {
          uint32_t sc = lds4(ring + (uint32_t)(slot * R::kStage + kv * R::kHalf +
                                               32 * R::kUnits + 4 * u));
          const int n = cv.end - t0;   // attended tokens of the unit, from its first
          if (n < 4) sc = n <= 0 ? 0u : sc & ((1u << (8 * n)) - 1u);
          if (kv == 1) {
            const uint32_t b = nan_bytes(sc);
            if (b) {
              sc &= ~((b >> 7) * 0xffu);
              nan = ((b >> 7) & 1u) | ((b >> 14) & 2u) | ((b >> 21) & 4u) | ((b >> 28) & 8u);
            }
          }
          e4m3x4_to_f16x2x2(sc, s01, s23);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t f[8];
          if constexpr (kFour) {
            const uint2 w = lds8(src + i * (R::kUnits * 8));
            uint32_t lo[4], hi[4];
            e2m1x8_to_f16x2(w.x, lo);
            e2m1x8_to_f16x2(w.y, hi);
            const uint32_t s = i < 2 ? s01 : s23;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[e] = (i & 1) ? hmul2_hi(lo[e], s) : hmul2_lo(lo[e], s);
              f[4 + e] = (i & 1) ? hmul2_hi(hi[e], s) : hmul2_lo(hi[e], s);
            }
          } else {
            uint4 w = lds16(src + i * (R::kUnits * 16));
            if (kv == 1 && (nan_bytes(w.x) | nan_bytes(w.y) | nan_bytes(w.z) | nan_bytes(w.w))) {
              nan |= 1u << i;
              w = make_uint4(0u, 0u, 0u, 0u);
            }
            e4m3x4_to_f16x2x2(w.x, f[0], f[1]);
            e4m3x4_to_f16x2x2(w.y, f[2], f[3]);
            e4m3x4_to_f16x2x2(w.z, f[4], f[5]);
            e4m3x4_to_f16x2x2(w.w, f[6], f[7]);
          }
          const uint32_t row = dst + (uint32_t)i * 128u;
          const uint32_t sw = (uint32_t)((4 * ua + i) & 7);
          const uint32_t ca = row + ((((uint32_t)(2 * g) & 7u) ^ sw) << 4);
          const uint32_t cb = row + ((((uint32_t)(2 * g + 1) & 7u) ^ sw) << 4);
          if (turn) {
            sts16(cb, f[4], f[5], f[6], f[7]);
            sts16(ca, f[0], f[1], f[2], f[3]);
          } else {
            sts16(ca, f[0], f[1], f[2], f[3]);
            sts16(cb, f[4], f[5], f[6], f[7]);
          }
        }
      }
      // ---- the stage's tag
      const uint32_t bad = ((bads >> slot) & 1u) ? 0xfu : 0u;
      if constexpr (D == 128) {   // a warp's units: 16 rows
        const int sh = 4 * (ua & 3);
        const uint32_t m = __reduce_or_sync(0xffffffffu, (bad << sh) | (nan << (16 + sh)));
        if (lane == 0) {
          uint16_t* const w = reinterpret_cast<uint16_t*>(c.tag[st].mask) + (warp - kLoaders);
          w[0] = (uint16_t)m;
          w[4] = (uint16_t)(m >> 16);
        }
      } else {                    // 32 rows, of V's warps
        const int sh = 4 * (ua & 7);
        const uint32_t mb = __reduce_or_sync(0xffffffffu, bad << sh);
        const uint32_t mn = __reduce_or_sync(0xffffffffu, nan << sh);
        if (lane == 0 && part0 == 1) {
          c.tag[st].mask[(warp - kLoaders) & 1] = mb;
          c.tag[st].mask[2 + ((warp - kLoaders) & 1)] = mn;
        }
      }
      if (x == 0) {
        const int nkt = cv.nkt(), klo = cv.lo / kKeys, n = cv.k1 - cv.k0, i = cv.k - cv.k0;
        const bool alt = ntok_b == 0;
        const int nkt_a = alt ? nkt : (cv.T - cv.L + (int)(w2 * cv.pr) + ntok_a - 1) / kKeys + 1;
        int f = (first ? kFirst : 0) | (cv.k == cv.k1 - 1 ? kLast : 0) | (alt ? kAlt : 0) |
                (cv.k0 == klo ? kBegins : 0);
        if (alt) {
          f |= (i & 1) ? kActB : kActA;
          if (i == 0) f |= kFirstA;
          if (i == 1) f |= kFirstB;
          if (i == ((n - 1) & ~1)) f |= kLastA;
          if (n >= 2) f |= kHasB;
          if (n >= 2 && i == ((n - 2) | 1)) f |= kLastB;
        } else {
          f |= kActB | (cv.k < nkt_a ? kActA : 0);
          if (i == 0) f |= kFirstB | kFirstA;
          if (cv.k == min(cv.k1, nkt_a) - 1) f |= kLastA;
          if (i == n - 1) f |= kLastB;
        }
        if (cv.k0 == klo && cv.k1 >= nkt_a) f |= kWholeA;
        if (cv.k0 == klo && cv.k1 == nkt) f |= kWholeB;
        Tag& tg = c.tag[st];
        tg.flags = f;
        tg.kt = cv.k;
        tg.h = cv.h;
        tg.q0 = q0;
        tg.ntok_a = ntok_a;
        tg.ntok_b = ntok_b;
        tg.p0 = cv.T - cv.L + (int)(w2 * cv.pr);
        tg.lo = cv.lo;
        tg.nkt_a = nkt_a;
        tg.nkt = nkt;
        tg.i0 = cv.i0;
        tg.len = cv.length();
      }
      fence_proxy_async_smem();   // the operands, before the tensor core reads them
      mbar_arrive(smem_u32(&c.full[st]));
      // ---- the copies of the stage that takes this one's place in the ring
      if (!ld.done) {
        issue(slot, ent);
        ent = entry(ld);
      }
      commit_copies();
      if (++slot == R::kRing) slot = 0;
      if (++st == S) {
        st = 0;
        ph ^= 1u;
      }
      cv.advance(a);
    }
    if (ok && wait_warp(c.empty[st], ph ^ 1u) && wait_warp(c.seen[st], ph ^ 1u)) {
      if (x == 0) c.tag[st].flags = kStop;
      mbar_arrive(smem_u32(&c.full[st]));
    } else if (lane == 0) {
      give_up();
    }
    wait_copies<0>();   // nothing lands in shared memory after the block's end
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ========================= softmax =========================
    const int tile = warp >> 2, wq = warp & 3;
    const int r = tid & 127;
    const uint32_t trow = tmem + ((uint32_t)(32 * wq) << 16);
    const uint32_t tcol = trow + (uint32_t)(256 * tile);
    unsigned long long* const tb = c.tile[tile];
    const int act = tile ? kActB : kActA, lastbit = tile ? kLastB : kLastA;
    const int tok_r = r / a.G;
    int ntok = 0, p0 = 0, prow = -1;
    bool busy = false;             // some row of this warp is a row
    float factor = 0.f, m_used = -INFINITY, l = 0.f;
    bool poison = false;
    bool ok = true;
    int st = 0, nt = 0, nb_alt = 0;
    uint32_t ph = 0u;
    while (true) {
      if (!wait_warp(c.full[st], ph)) {
        ok = false;
        break;
      }
      const Tag& tg = c.tag[st];
      const int flags = tg.flags, kt = tg.kt;
      if (flags & kStop) break;
      const uint4 mk = *reinterpret_cast<const uint4*>(tg.mask);
      const int h = tg.h, q0 = tg.q0, tag_lo = tg.lo;
      const int nkt_t = tile ? tg.nkt : tg.nkt_a;
      const long long i0 = tg.i0, line = tg.len;
      if (flags & kFirst) {
        const bool other = tile == 1 && !(flags & kAlt);   // rows of the second tile
        ntok = other ? tg.ntok_b : tg.ntok_a;
        p0 = tg.p0 + (other ? a.BM : 0);
        const bool valid = r < a.BM * a.G && tok_r < ntok;
        prow = valid ? p0 + tok_r : -1;
        busy = 32 * wq < ntok * a.G;
        factor = c.factor[st][other ? 1 : 0][r];
        m_used = -INFINITY;
        l = 0.f;
        poison = false;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.seen[st]));   // the tag is read
      if (++st == S) {
        st = 0;
        ph ^= 1u;
      }
      if (!(flags & act)) continue;
      if (!wait_warp(tb[kSFull], (uint32_t)nt & 1u)) {
        ok = false;
        break;
      }
      if (busy) {
        tc_fence_after();
        uint32_t sr[kKeys];
        tmem_ld32(tcol, *reinterpret_cast<uint32_t(*)[32]>(sr));
        tmem_ld32(tcol + 32, *reinterpret_cast<uint32_t(*)[32]>(sr + 32));
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(smem_u32(&tb[kSFree]));
        const int t0 = kt * kKeys;
        // P = 2^(s f - mu): one packed FFMA per two scores, one ex2 per score,
        // rounded to binary16; its sum in fp32 over the rounded values that O
        // sums, so that the rounding cancels where one key dominates
        uint32_t pk[kKeys / 2];
        auto p_pass = [&](float f, float mu) -> float {
          float sum[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] = 0.f;
#pragma unroll
          for (int e = 0; e < kKeys / 2; ++e) {
            float x0 = __uint_as_float(sr[2 * e]), x1 = __uint_as_float(sr[2 * e + 1]);
            ffma2(x0, x1, f, -mu);
            pk[e] = pack2<false>(ex2_approx(x0), ex2_approx(x1));
            sum[e & 7] = add_pair16<false>(sum[e & 7], pk[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] += sum[e + 4];
          return (sum[0] + sum[1]) + (sum[2] + sum[3]);
        };
        // A stage that all rows attend to needs no mask, and once the row has a
        // reference no maximum either: every P is at most their sum, so a sum of
        // at most 2^kTop shows that the reference stays.
        const bool plain = t0 + kKeys - 1 <= p0 && (mk.x | mk.y | mk.z | mk.w) == 0u &&
                           (a.window == 0 || (long long)t0 > (long long)p0 + ntok - 1 - a.window);
        const bool raw = plain && factor > 0.f;
        const bool guess = raw && m_used != -INFINITY;
        float alpha = 1.f, ssum = 0.f;
        if (guess) ssum = p_pass(factor, m_used);
        if (!guess || !(ssum <= kTopPow)) {
          float mx8[8], f = 1.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) mx8[e] = -INFINITY;
          if (raw) {
#pragma unroll
            for (int e = 0; e < kKeys / 2; ++e)
              mx8[e & 7] = max3f(mx8[e & 7], __uint_as_float(sr[2 * e]),
                                 __uint_as_float(sr[2 * e + 1]));
            f = factor;
          } else {
            // the keys this row attends to, a bit each
            uint64_t live = 0ull;
            if (prow >= t0) {
              const int hi = min(prow - t0, kKeys - 1);
              live = ~0ull >> (63 - hi);
              const long long first = (long long)prow - a.window + 1 - t0;
              if (a.window > 0 && first > 0) live = first > 63 ? 0ull : live & (~0ull << first);
              live &= ~(((uint64_t)mk.y << 32) | mk.x);
              poison = poison || (live & (((uint64_t)mk.w << 32) | mk.z)) != 0ull;
            }
            const uint32_t half[2] = {(uint32_t)live, (uint32_t)(live >> 32)};
#pragma unroll
            for (int e = 0; e < kKeys / 2; ++e) {
              float v[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int t = 2 * e + k;
                v[k] = ((half[t >> 5] >> (t & 31)) & 1u)
                           ? __uint_as_float(sr[t]) * factor : -INFINITY;
                sr[t] = __float_as_uint(v[k]);
              }
              mx8[e & 7] = max3f(mx8[e & 7], v[0], v[1]);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) mx8[e] = fmaxf(mx8[e], mx8[e + 4]);
          float mx = fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3]));
          if (raw) mx *= factor;
          bool moved = false;
          if (mx > m_used + kTop) {   // the exponentials' reference moves
            const float m_new = mx - kShift;
            if (m_used != -INFINITY) alpha = ex2_approx(m_used - m_new);
            m_used = m_new;
            moved = true;
          }
          if (!guess || moved) ssum = p_pass(f, m_used == -INFINITY ? 0.f : m_used);
        }
        l = l * alpha + ssum;
        // the P region's previous use is done: its product had completed before
        // these scores were issued
        tc_fence_after();
        __syncwarp();   // the collective stores and loads below take the whole warp
        tmem_st32(tcol + 64u + 32u * (uint32_t)(nt & 1), pk);
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
          // O rescaled once the previous stage's product is done
          if (nt >= 1 && !wait_warp(tb[kPEmpty + ((nt - 1) & 1)], (uint32_t)((nt - 1) >> 1) & 1u)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < D; cc += 32) {
            uint32_t o[32];
            tmem_ld32(tcol + 128u + (uint32_t)cc, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(tcol + 128u + (uint32_t)cc, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
      } else {
        // no row here: this warp's lanes of P and O hold anything, and nobody
        // reads them
        mbar_arrive(smem_u32(&tb[kSFree]));
      }
      mbar_arrive(smem_u32(&tb[kPFull + (nt & 1)]));
      if (flags & lastbit) {
        // ---- the part's end
        if (!wait_warp(tb[kPEmpty + (nt & 1)], (uint32_t)(nt >> 1) & 1u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (poison) l = __uint_as_float(0x7fffffffu);
        if ((flags & kAlt) && tile == 1) {
          // the same rows as tile A, the other stages: its warps join the two
          c.ml[r][0] = m_used;
          c.ml[r][1] = l;
          tc_fence_before();
          mbar_arrive(smem_u32(&c.bdone));
        } else {
          float wa = 1.f, wb = 0.f;
          const bool join = (flags & (kAlt | kHasB)) == (kAlt | kHasB);
          if (join) {
            if (!wait_warp(c.bdone, (uint32_t)nb_alt & 1u)) {
              ok = false;
              break;
            }
            ++nb_alt;
            tc_fence_after();
            const float mb = c.ml[r][0], lb = c.ml[r][1];
            const float m = fmaxf(m_used, mb), base = m == -INFINITY ? 0.f : m;
            wa = ex2_approx(m_used - base);
            wb = ex2_approx(mb - base);
            l = l * wa + lb * wb;
            m_used = m;
          }
          const bool whole = (flags & (tile ? kWholeB : kWholeA)) != 0;
          const float mul = whole ? (l == 0.f ? 0.f : a.v_scale / l) : 1.f;
          wa *= mul;
          wb *= mul;
          uint16_t* const orow =
              a.out + ((size_t)(q0 + (tile ? a.BM : 0) + (prow >= 0 ? tok_r : 0)) * a.Hq +
                       (size_t)h * a.G + r % a.G) * D;
          float* const rec =
              a.ws_rec + (((size_t)blockIdx.x * 2 + ((flags & kBegins) ? 1 : 0)) * 2 + tile) *
                             rec_floats(D);
          if (busy) {
#pragma unroll 1
            for (int cc = 0; cc < D; cc += 32) {
              uint32_t o[32];
              tmem_ld32(tcol + 128u + (uint32_t)cc, o);
              if (join) {
                uint32_t o2[32];
                tmem_ld32(trow + 256u + 128u + (uint32_t)cc, o2);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  o[e] = __float_as_uint(__uint_as_float(o[e]) * wa + __uint_as_float(o2[e]) * wb);
              } else {
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * wa);
              }
              if (prow >= 0 && whole) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint32_t w[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    w[k] = pack2<kBF16>(__uint_as_float(o[8 * e + 2 * k]),
                                        __uint_as_float(o[8 * e + 2 * k + 1]));
                  *reinterpret_cast<uint4*>(orow + cc + 8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
                }
              } else if (prow >= 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  *reinterpret_cast<uint4*>(rec + (size_t)r * D + cc + 4 * e) =
                      make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
              }
              __syncwarp();
            }
          }
          tc_fence_before();
          mbar_arrive(smem_u32(&tb[kOFree]));
          if (join) mbar_arrive(smem_u32(&c.tile[1][kOFree]));
          if (!whole) {
            if (prow >= 0) {
              rec[(size_t)kTileRows * D + r] = m_used;
              rec[(size_t)kTileRows * (D + 1) + r] = l;
            }
            group_sync(1 + tile);
            // the records of this tile: the blocks that hold stages of it
            if (wq == 0) {
              int f = blockIdx.x, e = blockIdx.x;
              while (f > 0 && c.bound[f] > i0) --f;
              while (e + 1 < nb && c.bound[e + 1] < i0 + line) ++e;
              int n = 0, end = f;
              for (int b0 = f; b0 <= e; b0 += 32) {
                const int b = b0 + lane;
                bool in = false, begins = false;
                if (b <= e) {
                  const int s0 = stage_at(c.bound[b] - i0, tag_lo, nkt_t);
                  in = s0 < stage_at(c.bound[b + 1] - i0, tag_lo, nkt_t);
                  begins = s0 == tag_lo / kKeys;
                }
                const uint32_t all = __ballot_sync(0xffffffffu, in);
                if (in) c.parts[tile][n + __popc(all & ((1u << lane) - 1u))] =
                    (uint16_t)(b * 2 + (begins ? 1 : 0));
                n += __popc(all);
                if (all) end = b0 + 31 - __clz(all);
              }
              if (lane == 0) {
                c.nparts[tile] = n;
                // releases this tile's record (ordered before by the barrier),
                // acquires those counted before it
                uint32_t* const cnt = a.ws_count + 2 * end + tile;
                const bool last = atom_add_acq_rel_gpu(cnt, 1u) + 1u == (uint32_t)n;
                if (last) *cnt = 0u;   // ready for the next call
                c.last[tile] = last ? 1 : 0;
              }
            }
            group_sync(1 + tile);
            if (c.last[tile]) {
              // ---- the last record: join them all, in the order of the keys
              constexpr int kLanes = D / 4, kRows = 128 / kLanes;
              const int n = c.nparts[tile], rows = ntok * a.G, col = 4 * (r % kLanes);
              for (int rr = r / kLanes; rr < rows; rr += kRows) {
                float m = -INFINITY, ls = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k0 = 0; k0 < n; k0 += 4) {
                  float4 v[4];
                  float pm[4], pl[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const float* p = a.ws_rec +
                                     ((size_t)c.parts[tile][min(k0 + k, n - 1)] * 2 + tile) *
                                         rec_floats(D);
                    v[k] = __ldcg(reinterpret_cast<const float4*>(p + (size_t)rr * D + col));
                    pm[k] = __ldcg(p + (size_t)kTileRows * D + rr);
                    pl[k] = __ldcg(p + (size_t)kTileRows * (D + 1) + rr);
                  }
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    if (k0 + k >= n) break;
                    const float mn = fmaxf(m, pm[k]), base = mn == -INFINITY ? 0.f : mn;
                    const float x = ex2_approx(m - base), y = ex2_approx(pm[k] - base);
                    m = mn;
                    ls = ls * x + pl[k] * y;
                    acc.x = acc.x * x + v[k].x * y;
                    acc.y = acc.y * x + v[k].y * y;
                    acc.z = acc.z * x + v[k].z * y;
                    acc.w = acc.w * x + v[k].w * y;
                  }
                }
                const float mulr = ls == 0.f ? 0.f : a.v_scale / ls;
                const int tok = rr / a.G;
                uint16_t* const dst =
                    a.out + ((size_t)(q0 + (tile ? a.BM : 0) + tok) * a.Hq + (size_t)h * a.G +
                             (rr - tok * a.G)) * D + col;
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<kBF16>(acc.x * mulr, acc.y * mulr),
                                                            pack2<kBF16>(acc.z * mulr, acc.w * mulr));
              }
            }
          }
        }
      }
      ++nt;
    }
    if (!ok && lane == 0) give_up();
  }

  // ---- every product has completed: release the tensor memory
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kAlloc) tmem_dealloc(tmem, 512);
}

inline int check_prefill_shape(int Hq, int H, int D) {
  if (Hq <= 0 || H <= 0 || Hq % H != 0) return PA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return PA_ERR_UNSUPPORTED;
  if (Hq / H > 16) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

inline int prefill_quant_grid(int* grid) {
  DeviceInfo di;
  if (int rc = current_device_info(&di)) return rc;
  *grid = di.sm_count < kMaxGrid ? di.sm_count : kMaxGrid;
  return PA_OK;
}

inline size_t prefill_quant_bytes(int D, int grid) {
  return PA_PREFILL_QUANT_COUNTERS + (size_t)grid * 4 * rec_floats(D) * sizeof(float);
}
static_assert(2 * kMaxGrid * sizeof(uint32_t) <= PA_PREFILL_QUANT_COUNTERS, "two counters a block");

// The kernels' opt-in to their shared memory, once a device.
constexpr int kMaxDevices = 64;

template <int D, bool kBF16, bool kFour>
int launch_prefill_quant(const Args& a, int grid, int device, cudaStream_t s) {
  static std::mutex mu;
  static bool ready[kMaxDevices];
  const auto kern = prefill_quant_kernel<D, kBF16, kFour>;
  constexpr size_t smem = smem_bytes<D, kFour>();
  static_assert(smem <= 227 * 1024, "a block's shared memory");
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[device]) {
      cudaError_t e =
          cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      cudaFuncAttributes at{};
      if (!e) e = cudaFuncGetAttributes(&at, kern);
      if (e) return launch_status(e, "cudaFuncSetAttribute (quantized prefill)");
      // the roles re-divide the launch's registers, which the increases wait for
      if (at.numRegs != 128) return PA_ERR_UNSUPPORTED;
      ready[device] = true;
    }
  }
  clear_stale_error();
  return launch_status(launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads), smem, s, a),
                       "quantized prefill launch");
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
  if (int rc = check_prefill_shape(num_q_heads, num_kv_heads, head_dim)) return rc;
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
  DeviceInfo di;
  if (int rc = current_device_info(&di)) return rc;
  int grid = 0;
  if (int rc = prefill_quant_grid(&grid)) return rc;
  if (workspace_bytes < prefill_quant_bytes(head_dim, grid)) return PA_ERR_WORKSPACE;
  Args a{};
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.kc = static_cast<const uint8_t*>(k_cache);
  a.vc = static_cast<const uint8_t*>(v_cache);
  a.bt = block_tables;
  a.seq_lens = seq_lens;
  a.query_start = query_start;
  a.ws_count = static_cast<uint32_t*>(workspace);
  a.ws_rec = reinterpret_cast<float*>(static_cast<char*>(workspace) + PA_PREFILL_QUANT_COUNTERS);
  a.err = err_word;
  a.num_blocks = num_blocks;
  a.total_q = total_q;
  a.num_seqs = num_seqs;
  a.stride = table_stride;
  a.Hq = num_q_heads;
  a.H = num_kv_heads;
  a.G = num_q_heads / num_kv_heads;
  a.BM = kTileRows / a.G;
  a.log2B = ilog2(block_size);
  a.window = window;
  a.scale_log2 = scale * k_scale * 1.4426950408889634f;
  a.v_scale = v_scale;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = q_dtype == PA_BF16;
  if (head_dim == 64)
    return bf16 ? launch_prefill_quant<64, true, kFour>(a, grid, di.device, s)
                : launch_prefill_quant<64, false, kFour>(a, grid, di.device, s);
  return bf16 ? launch_prefill_quant<128, true, kFour>(a, grid, di.device, s)
              : launch_prefill_quant<128, false, kFour>(a, grid, di.device, s);
}

}  // namespace

}  // namespace pa
