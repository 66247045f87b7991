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
// The weights are one binary16 value each (2^-11), as the chunks over 16-bit pools hold
// one value of the query's type: binary16 outputs are 2.8e-4 off 64 bits in norm (2.1e-4
// is their own rounding), bfloat16 ones 1.7e-3 with either.  A pair of values, as the
// 4-bit decode has, takes a second product and, tensor memory being full (64 columns of
// scores, 64 of weights, 128 of values a tile of head_dim 128), leaves one place for
// weights instead of two.  Built and measured, us for the pair / for one value: 16 chunks of
// 512 over 4 bits 640 / 486, the 32 K prompt 1,289 / 993, 32 verified contexts 749 / 600,
// chunks of 400 and head_dim 64 151 / 130.
//
// Roles of a block of 20 warps, one block an SM:
//  * warp 18 walks the block's share of the work and writes a tag for every stage
//    of 64 keys: what is to be done with it, and where its blocks lie.
//  * warps 8-11 (K) and 12-15 (V), 16 keys each, fetch the codes as they lie in
//    the pool into a ring of their own, some stages ahead (16-byte asynchronous
//    copies: a TMA copy cost its issuing warp 200 to 300 cycles, and a stage of
//    16-token blocks takes eight), and turn them into 16-bit operands with the
//    128-byte swizzle.  With a part's first stage they bring the query rows of
//    tile A and of tile B in, whole rows a copy (a row a thread took 7 us a part),
//    and turn them into binary16 where they lie.
//  * warps 16 and 17 (a tile each): S = Q K^T of a stage;
//  * warp 19 (both tiles): O += P V, P from tensor memory.
//  * warps 0-3 (tile A) and 4-7 (tile B): thread r owns row r, tensor memory
//    lane r.  It reads its scores, masks them, writes P = 2^(s - m) and keeps
//    the row's sum; m moves only when a weight would pass 2^kTop, and then the
//    row of O is rescaled in tensor memory.
// A pair without a second tile gives its stages to the tiles in turn: both hold
// the same rows and end with partial results, which tile A's warps join.
//
// The split.  The pairs of all sequences and KV heads, in that order, are a line
// on which a pair is `start` + (its attended tokens) long; it is cut into equal
// shares, one a block.  A pair cut between blocks leaves one record (O, m, l) a
// tile and block in the workspace, and the last block to count its record joins
// them, always in the order of the keys: no block waits for another, and the
// result depends on nobody's speed.
//
// What bounds it.  Products at the tensor cores' rate are the floor of long chunks; the
// conversion comes before it: a stage is one chain a warp (wait for the place, codes
// from shared memory, conversion, stores, fence, arrival, the next copies) of some
// 1,700 cycles, and beside two query tiles of 32 KB (head_dim 128) three stages fit,
// or six of head_dim 64.  Measured: 1,024 new tokens at 31,744 of an E4M3 cache, 64
// query and 8 KV heads of 128, 994 us (1,090 TFLOP/s); 16 chunks of 512 over 4 bits,
// 32 and 8 heads, 488 us (968 TFLOP/s); 32 contexts of 16 to 33 K tokens over 4 bits
// with four new tokens each, 64 and 8 heads, 601 us (1.6 TB/s: a quarter of the
// rows are in use); 7 ragged chunks of up to 277 with a window of 512, 76 us.
#pragma once

#include <cmath>
#include <mutex>

#include "pa_fp4.cuh"
#include "pa_host.h"

namespace pa {

namespace {

constexpr int kKeys = 64;                 // of a stage
constexpr int kConvert = 8;               // first conversion warp
constexpr int kIssue = 16;                // warps 16 and 17
constexpr int kTagger = 18;
constexpr int kValues = 19;
constexpr int kThreads = 640;
constexpr int kMaxGrid = 256;
constexpr uint32_t kWaitCycles = 3800000000u;   // about 2 s, as every wait of the library
// A pair's start and end cost what this many tokens do.  bfloat16 queries, which are
// scaled, us with 128 / 256 / 384: 16 chunks of 512 over 4 bits 565 / 516 / 485, 64
// sequences over E4M3 157 / 147 / 142, 4 prompts of 2,048 230 / 212 / 203, 7 chunks with
// a window 77 / 78 / 79, 20 of head_dim 64 159 / 159 / 157.  Binary16 ones: 534 / 493 /
// 491, 144 / 138 / 137, 207 / 191 / 195, 74 / 76 / 77, 130 / 130 / 132: short pairs
// decided, the long ones would take 256.
constexpr int kStart[2] = {128, 384};   // binary16, bfloat16
// Small batches take a block for every kLeast of the line (256 and 768: within 1%).
constexpr int kLeast = 384;
// The exponentials' reference is a maximum less kShift when it is set and stays
// until a weight would pass 2^kTop: binary16 holds weights down to 2^-14 - kShift
// of the maximum with all their bits.
constexpr float kShift = 7.f, kTop = 15.f, kTopPow = 32768.f;
// Registers of the roles: softmax, conversion, the others (5 x 96 a thread; 8 to 52
// bytes a thread are spilled).
constexpr int kRegsLaunch = 96;
constexpr int kRegsSoftmax = 136, kRegsConvert = 72, kRegsOther = 64;
static_assert(2 * kRegsSoftmax + 2 * kRegsConvert + kRegsOther == 5 * kRegsLaunch,
              "the launch's registers");

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
  int start;                // what a pair's start and end cost, in tokens
  int few;                  // which of the two kernels take sequences of few rows
  uint32_t* few_count;      // [grid], zero between calls
  float* few_rec;           // [grid][2] records of few_rec_floats(D)
};
// kFewNone: this kernel takes all sequences; kFewBoth: pa_prefill_few.cuh's those of
// few rows; kFewOnly: it takes all
enum : int { kFewNone, kFewBoth, kFewOnly };
constexpr int kFewRows = 16;

constexpr int kTileRows = 128;
// o[D / 4][128][4] (a warp's 32 rows lie together), m[128], l[128]
__host__ __device__ constexpr size_t rec_floats(int D) { return (size_t)kTileRows * (D + 2); }

// A conversion warp's 16 rows of K or V: the rows' codes one after the other, then
// a 4-bit pool's scales, four rows (a quad) at a time as they lie in the pool.
template <int D, bool kFour>
struct Raw {
  static constexpr int kRowBytes = kFour ? D / 2 : D;
  static constexpr int kCodes = 16 * kRowBytes;
  static constexpr int kWarp = kCodes + (kFour ? D : 0);
  static constexpr int kStage = 8 * kWarp;
  static constexpr int kRing = D == 64 ? 6 : (kFour ? 5 : 3);      // stages in flight
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
  kHasB = 8192,
  kEdge = 1 << 15,                // some rows hold no data
  kMarked = 1 << 16               // some bit of `mask` is set
};

// What is to be known about a stage, beside its keys.
struct Tag {
  int flags, kt;
  uint32_t rows[2];                 // (kEdge) bits of keys: rows that hold data
  uint32_t mask[4];                 // (kMarked) left out (2 words), NaN value rows (2 words)
  // of the part, with a tile's first stage
  int h, q0, p0, lo;                // q0: tile A's first q row; p0: its position; lo: first
                                    // attended token
  int ntok_a, ntok_b, nkt_a, nkt;   // tokens of the tiles, ends of their stages
  long long i0, len;                // the pair's place on the line, its length there
  int part, pad[3];                 // its number in this block
  // where the stage's pieces (min(B, 64) rows of one block) begin in the pools, or
  // -1: not to be read
  long long at[kKeys / 4];
};

constexpr int kShare = 6;   // a tile's arrivals on a stage's `empty`
constexpr int kBatch = 4;   // tags written together

template <int S, int kRing>
struct Control {
  // tags are written kBatch at a time, so far ahead that the fetches, kRing stages
  // ahead of the conversion, find theirs
  static constexpr int kAhead = kRing + 2 * kBatch;
  static constexpr int kTags = S + kAhead;

  unsigned long long full[S], empty[S], tfull[kAhead], tempty[kAhead];
  unsigned long long qempty, bdone, done[3];
  unsigned long long tile[2][8];    // s full, s free, p full[2], p empty[2], o free
  unsigned long long met[2];        // a tile's softmax warps
  alignas(16) Tag tag[kTags];
  // of a part's rows: what scores are multiplied by; before the first part, the
  // line before each thread's run of sequences
  union {
    float factor[S + 1][2][kTileRows];
    long long run_pref[kThreads];
  };
  float ml[kTileRows][2];           // tile B's m and l, of a pair in turn
  int4 scores[2][4];                // of a tile's score products: flags, stage, slot, tag
  long long warp_tot[kThreads / 32];
  long long bound[kMaxGrid + 1];
  uint16_t parts[2][kMaxGrid];      // of a cut tile: its records
  float join[2][kTileRows][2];      // and its rows' maxima, and factors of the sums
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
         Raw<D, kFour>::kRing * Raw<D, kFour>::kStage + sizeof(Control<Tiles<D>::kStages, Raw<D, kFour>::kRing>);
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

// 16 bytes from global to shared memory, past L1
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("{\n\t.reg .b64 s;\n\tmbarrier.arrive.shared::cta.b64 s, [%0], %1;\n\t}" ::"r"(bar),
               "r"(n)
               : "memory");
}
// One lane of the warp, which the compiler knows to be one.  tcgen05 instructions
// stand behind this in code that all lanes reach: behind `lane == 0` each of them
// is given a choice of lane and moves of its operands of its own (125 cycles for a
// product's issue).
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0u;
}
// once for the warp, behind what its lanes did
__device__ __forceinline__ void warp_arrive(unsigned long long& bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bar));
}
__device__ __forceinline__ int ilog2_device(int x) { return 31 - __clz(x); }
// bytes of E4M3 codes that are NaN: 0x80 in their place
__device__ __forceinline__ uint32_t nan_bytes(uint32_t x) {
  return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Sequence i: its rows of q and its length; false (no tokens then) where they
// contradict each other or the table.
__device__ __forceinline__ bool load_any(const Args& a, int i, int& q0, int& L, int& T) {
  const int s0 = __ldg(a.query_start + i), s1 = __ldg(a.query_start + i + 1);
  T = __ldg(a.seq_lens + i);
  const long long n = (long long)s1 - s0;
  const bool ok = s0 >= 0 && n >= 0 && s1 <= a.total_q && T >= 0 &&
                  (long long)T <= ((long long)a.stride << a.log2B) && n <= T;
  q0 = s0;
  L = ok ? (int)n : 0;
  return ok;
}

// Of those, what the kernel with tiles of 128 rows takes.
__device__ __forceinline__ bool load_seq(const Args& a, int i, int& q0, int& L, int& T) {
  const bool ok = load_any(a, i, q0, L, T);
  if (a.few == kFewBoth && (long long)L * a.G <= kFewRows) L = 0;
  return ok;
}

// The same by a whole warp, which goes on with one lane's words: lengths that change
// during the call then cannot part its lanes.
__device__ __forceinline__ void load_seq_warp(const Args& a, int i, int& q0, int& L, int& T) {
  load_seq(a, i, q0, L, T);
  q0 = __shfl_sync(0xffffffffu, q0, 0);
  L = __shfl_sync(0xffffffffu, L, 0);
  T = __shfl_sync(0xffffffffu, T, 0);
}

// Sequences that contradict themselves: reported, their rows cleared.
__device__ __forceinline__ void clear_bad(const Args& a, int D, int threads) {
  for (int i = blockIdx.x; i < a.num_seqs; i += gridDim.x) {
    int q0, L, T;
    if (load_any(a, i, q0, L, T)) continue;
    if (threadIdx.x == 0) set_error(a.err, PA_DEVERR_SEQ_LEN);
    const long long r0 = max(q0, 0);
    const long long r1 = min((long long)__ldg(a.query_start + i + 1), a.total_q);
    uint4* dst = reinterpret_cast<uint4*>(a.out + (size_t)r0 * a.Hq * D);
    for (long long e = threadIdx.x; e < (r1 - r0) * a.Hq * (D / 8); e += threads)
      dst[e] = make_uint4(0u, 0u, 0u, 0u);
  }
}

__device__ __forceinline__ int pairs_of(int L, const Args& a) {
  return (int)(((long long)L + 2 * a.BM - 1) / (2 * a.BM));
}

// The line's length of pairs 0 .. pr - 1 of a sequence with P of them (one KV
// head): pair j ends with token T - L + min(2 BM (j + 1), L) and begins with the
// first token its first row attends to.
__device__ __noinline__ long long line_before(long long pr, long long P, int L, int T,
                                                 const Args& a) {
  const long long base = (long long)T - L, w = 2 * a.BM;
  long long sum = a.start * pr;
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
// stands at `start`).
__device__ __forceinline__ int stage_at(long long at, int lo, int nkt, int start) {
  const long long r = at - start;
  if (r <= 0) return lo / kKeys;
  const long long k = (lo + r + kKeys - 1) / kKeys;
  return k < nkt ? (int)k : nkt;
}

// A place in a block's share of the line (a warp's).
struct Walk {
  int i, q0, L, T, P;          // sequence
  int h, pr, lo, end;          // pair: first attended token, end of the attended ones
  int k, k0, k1;               // stage; the stages of this block's part of the pair
  long long i0, u0, u1;        // the pair's place; the block's share
  bool done;

  __device__ __forceinline__ long long length(const Args& a) const {
    return (long long)a.start + end - lo;
  }
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
      k0 = stage_at(u0 - i0, lo, nkt(), a.start);
      k1 = stage_at(u1 - i0, lo, nkt(), a.start);
      k = k0;
      if (k0 < k1) return;
      next_pair(a);
    }
  }
  __device__ __forceinline__ void next_pair(const Args& a) {
    i0 += length(a);
    if (++pr < P) return;
    pr = 0;
    if (++h < a.H) return;
    h = 0;
    P = 0;
    while (P == 0 && ++i < a.num_seqs) {
      load_seq_warp(a, i, q0, L, T);
      P = pairs_of(L, a);
    }
  }
  // to place u0 of the line
  __device__ __forceinline__ void start(const Args& a, const long long* run_pref, int per,
                                        long long from, long long to) {
    u0 = from;
    u1 = to;
    done = false;
    int r = 0;   // the last run that starts at or before u0
#pragma unroll
    for (int b = 512; b > 0; b >>= 1)
      if (r + b < kThreads && run_pref[r + b] <= u0) r += b;
    long long rem = u0 - run_pref[r], one = 0;
    i = r * per;
    while (i < a.num_seqs) {
      load_seq_warp(a, i, q0, L, T);
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
  using C = Control<S, R::kRing>;
  C& c = *reinterpret_cast<C*>(smem_raw + (ring - raw0) + R::kRing * R::kStage);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      // the conversion warps: K's and V's, whose NaN the scores' softmax has to know
      mbar_init(smem_u32(&c.full[s]), 8);
      // per tile: K read, V read, and its four softmax warps have read the tag
      mbar_init(smem_u32(&c.empty[s]), 2 * kShare);
    }
    for (int s = 0; s < C::kAhead; ++s) {
      mbar_init(smem_u32(&c.tfull[s]), 1);       // the tag is written
      mbar_init(smem_u32(&c.tempty[s]), 8);      // its stage is converted
    }
    mbar_init(smem_u32(&c.qempty), 2);           // a commit of each score issuer
    mbar_init(smem_u32(&c.bdone), 4);            // tile B's warps
    for (int k = 0; k < 3; ++k) mbar_init(smem_u32(&c.done[k]), 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&c.tile[t][kSFull]), 2);        // the product, its record
      mbar_init(smem_u32(&c.tile[t][kSFree]), 4);        // the tile's warps
      for (int p = 0; p < 2; ++p) {
        mbar_init(smem_u32(&c.tile[t][kPFull + p]), 4);  // the same
        mbar_init(smem_u32(&c.tile[t][kPEmpty + p]), 1);
      }
      mbar_init(smem_u32(&c.tile[t][kOFree]), 4);
      mbar_init(smem_u32(&c.met[t]), 4);
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
  if (odd) clear_bad(a, D, kThreads);
  const long long nb = min((long long)gridDim.x, (total + kLeast - 1) / kLeast);
  if ((long long)blockIdx.x >= nb) return;
  if (tid <= nb) c.bound[tid] = total * tid / nb;
  if (warp == kTagger) {
    tmem_alloc(smem_u32(&c.tmem), 512);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  // (before the roles' registers are cut: it calls a function)
  Walk w;
  if (warp == kTagger) w.start(a, c.run_pref, per, c.bound[blockIdx.x], c.bound[blockIdx.x + 1]);

  // a wait whose outcome is the same in every lane of the warp (every wait stands in
  // line: it is kept short)
  auto wait_warp = [&](unsigned long long& bar, uint32_t parity) -> bool {
    const uint32_t at = smem_u32(&bar);
    if (__all_sync(0xffffffffu, mbar_try_wait(at, parity))) return true;
    const uint32_t t0 = (uint32_t)clock();
#pragma unroll 1
    while (!__all_sync(0xffffffffu, mbar_try_wait(at, parity)))
      if (c.abort != 0 || (uint32_t)clock() - t0 > kWaitCycles) return false;
    return true;
  };
  auto give_up = [&]() {   // by one thread: the other roles leave on the flag
    if (!c.abort) set_error(a.err, PA_DEVERR_TIMEOUT);
    c.abort = 1;
  };

  if (warp >= kIssue) {
    setmaxnreg_dec<kRegsOther>();
    if (warp < kTagger) {
      // ===================== score products of tile t =====================
      // S = Q K^T of the tile's next stage once its keys are there, its S buffer has
      // been read and the P region that its weights will go to is free.
      const int t = warp - kIssue;
      const int act = t == 0 ? kActA : kActB;
      constexpr uint32_t id_s = umma_idesc_f16(false, kTileRows, kKeys, false);
      unsigned long long* const tb = c.tile[t];
      const uint32_t tcol = tmem + (uint32_t)(256 * t);
      const uint64_t dq[2] = {umma_desc_sw128(qtiles, 16, 1024),
                              umma_desc_sw128(qtiles + (uint32_t)t * X::kQTile, 16, 1024)};
      int rt = 0, st = 0, tg = 0;     // scores issued, slots
      uint32_t ph = 0u;
      bool ok = true;
      auto wait = [&](unsigned long long& bar, uint32_t parity) {
        ok = ok && wait_warp(bar, parity);
        return ok;
      };
      while (true) {
        if (!wait(c.full[st], ph)) break;
        const int flags = c.tag[tg].flags;
        if (flags & (act | kStop)) {
          // the softmax has read the scores (and their record) before these
          if (rt >= 1 && !wait(tb[kSFree], (uint32_t)(rt - 1) & 1u)) break;
          if (flags & kStop) {
            if (lane == 0) {
              c.scores[t][rt & 3] = make_int4(flags, 0, 0, 0);
              mbar_arrive_n(smem_u32(&tb[kSFull]), 2);
            }
            break;
          }
          if (rt >= 2 && !wait(tb[kPEmpty + (rt & 1)], (uint32_t)((rt >> 1) - 1) & 1u)) break;
          if (lane == 0) {
            c.scores[t][rt & 3] = make_int4(flags, c.tag[tg].kt, st, tg);
            mbar_arrive(smem_u32(&tb[kSFull]));
          }
          tc_fence_after();
          const uint64_t da = dq[(flags & kAlt) ? 0 : 1];
          const uint64_t db = umma_desc_sw128(stages + (uint32_t)st * X::kStage, 16, 1024);
          if (elect()) {
            // K steps of 16 columns: 32 bytes on within a 64-column plane
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t o = (uint32_t)(ks & 3) * 32u, p = (uint32_t)(ks >> 2);
              umma_f16(tcol, da + ((p * X::kQPlane + o) >> 4), db + ((p * X::kPlane + o) >> 4),
                       id_s, ks > 0);
            }
            umma_commit(smem_u32(&tb[kSFull]));
            umma_commit(smem_u32(&c.empty[st]));   // K is read
            if (flags & kLast) umma_commit(smem_u32(&c.qempty));   // the queries are read
          }
          __syncwarp();
          ++rt;
        } else {   // not this tile's: all but the V share
          if (elect()) {
            mbar_arrive_n(smem_u32(&c.empty[st]), kShare - 1);
            if (flags & kLast) umma_commit(smem_u32(&c.qempty));
          }
          __syncwarp();
        }
        if (++st == S) {
          st = 0;
          ph ^= 1u;
        }
        if (++tg == C::kTags) tg = 0;
      }
      if (!ok && lane == 0) give_up();
      // every product has completed before the tensor memory is released
      if (elect()) umma_commit(smem_u32(&c.done[t]));
      __syncwarp();
      mbar_wait_bounded(smem_u32(&c.done[t]), 0u, nullptr);
    } else if (warp == kValues) {
      // ===================== O += P V of both tiles =====================
      // Each tile's stages in order; of the two, whichever has its weights written.
      constexpr uint32_t id_o = umma_idesc_f16(false, kTileRows, D, true);
      struct Cursor {
        int n, ni, st, tg;   // products issued, parts begun, slots
        uint32_t ph;
        bool done;
      };
      Cursor cur[2] = {{0, 0, 0, 0, 0u, false}, {0, 0, 0, 0, 0u, false}};
      auto ready = [&](unsigned long long& bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_test(smem_u32(&bar), parity)) != 0;
      };
      auto step = [&](int t, Cursor& k) -> bool {   // whether the tile went a stage on
        if (k.done || !ready(c.full[k.st], k.ph)) return false;
        const int flags = c.tag[k.tg].flags;
        unsigned long long* const tb = c.tile[t];
        if (flags & kStop) {
          k.done = true;
          return true;
        }
        if (flags & (t == 0 ? kActA : kActB)) {
          const bool first = (flags & (t == 0 ? kFirstA : kFirstB)) != 0;
          if (!ready(tb[kPFull + (k.n & 1)], (uint32_t)(k.n >> 1) & 1u)) return false;
          if (first && k.ni > 0 && !ready(tb[kOFree], (uint32_t)(k.ni - 1) & 1u)) return false;
          if (first) ++k.ni;
          tc_fence_after();
          // V (64 keys x D) MN-major: 64-column planes kPlane apart, groups of 8
          // keys 1024 bytes apart; 16 keys a step, 8 columns of P
          const uint32_t tcol = tmem + (uint32_t)(256 * t);
          const uint64_t dv = umma_desc_sw128(stages + (uint32_t)k.st * X::kStage + X::kPart,
                                              X::kPlane, 1024);
          const uint32_t p = tcol + 64u + 32u * (uint32_t)(k.n & 1);
          if (elect()) {
#pragma unroll
            for (int e = 0; e < kKeys / 16; ++e)
              umma_tmem_a(tcol + 128u, p + 8u * e, dv + ((uint32_t)e * 2048u >> 4), id_o,
                          !first || e > 0);
            umma_commit(smem_u32(&tb[kPEmpty + (k.n & 1)]));
            umma_commit(smem_u32(&c.empty[k.st]));   // V is read
          }
          __syncwarp();
          ++k.n;
        } else if (lane == 0) {
          mbar_arrive(smem_u32(&c.empty[k.st]));
        }
        if (++k.st == S) {
          k.st = 0;
          k.ph ^= 1u;
        }
        if (++k.tg == C::kTags) k.tg = 0;
        return true;
      };
      long long t_last = clock64();
      while (!(cur[0].done && cur[1].done)) {
        const bool a0 = step(0, cur[0]), a1 = step(1, cur[1]);
        if (a0 || a1) {
          t_last = clock64();
        } else if (__any_sync(0xffffffffu,
                              c.abort != 0 || clock64() - t_last > kWaitLimitCycles)) {
          if (lane == 0) give_up();
          break;
        }
      }
      if (elect()) umma_commit(smem_u32(&c.done[2]));
      __syncwarp();
      mbar_wait_bounded(smem_u32(&c.done[2]), 0u, nullptr);
    } else if (warp == kTagger) {
      // ===================== tags =====================
      const int B = 1 << a.log2B;
      const int bs = min(B, kKeys), nblk = kKeys / bs;   // rows of a piece, pieces of a stage
      // bytes of a block, of a block's head, of a row of it
      const long long block_bytes = kFour ? (long long)a.H * B * fp4_row_bytes(D)
                                          : (long long)B * a.H * D;
      const int head_bytes = kFour ? B * fp4_row_bytes(D) : D;
      const int row_bytes = kFour ? D / 2 : a.H * D;
      // Tags of up to kBatch stages of a part together, a lane each, and a table
      // entry a lane (in kRounds rounds), which is loaded ahead of the wait for the
      // tags' places: value v is piece v % nblk of stage v / nblk
      constexpr int kRounds = kBatch * 16 / 32;
      const int lognblk = ilog2_device(nblk);
      int ents[kRounds];
      bool need[kRounds];
      bool begun = false;
      auto look = [&]() {
        if (!begun || w.k >= w.k1) {   // the first part, or the next
          if (begun) w.next_pair(a);
          begun = true;
          w.settle(a);
        }
#pragma unroll
        for (int u = 0; u < kRounds; ++u) {
          const int v = lane + 32 * u;
          const int k = w.k + (v >> lognblk);
          const int t = (int)((uint32_t)k * kKeys) + (v & (nblk - 1)) * bs;   // (k < k1: in range)
          // whether a row of it is attended to (an entry that is needed may hold anything)
          need[u] = !w.done && v < kBatch * nblk && k < w.k1 && t > w.lo - bs && t < w.end;
          ents[u] = need[u] ? __ldg(a.bt + (size_t)w.i * a.stride + (t >> a.log2B)) : -1;
        }
      };
      int ts = 0, tg = 0, parts = 0, part = 0, nkt_a = 0;
      uint32_t ph = 0u;
      bool ok = true;
      while (true) {
        look();
        const int m = w.done ? 1 : min(kBatch, w.k1 - w.k);   // stages of this batch
        for (int k = 0; k < m && ok; ++k) {
          const int b = ts + k;
          ok = wait_warp(c.tempty[b < C::kAhead ? b : b - C::kAhead],
                         (b < C::kAhead ? ph : ph ^ 1u) ^ 1u);
        }
        if (!ok) {
          if (lane == 0) give_up();
          break;
        }
        // this lane's stage of the batch, its tag and barrier
        const int k = lane < m ? lane : 0;
        const int tk = tg + k < C::kTags ? tg + k : tg + k - C::kTags;
        Tag& t = c.tag[tk];
        const int bk = ts + k < C::kAhead ? ts + k : ts + k - C::kAhead;
        if (w.done) {
          if (lane == 0) t.flags = kStop;
          warp_arrive(c.tfull[ts]);
          break;
        }
        uint32_t want[kRounds], got[kRounds];
#pragma unroll
        for (int u = 0; u < kRounds; ++u) {
          const int v = lane + 32 * u, ent = ents[u];
          const bool on = ent >= 0 && (long long)ent < a.num_blocks;
          if (need[u] && !on) set_error(a.err, PA_DEVERR_BLOCK_ID);
          want[u] = __ballot_sync(0xffffffffu, need[u]);
          got[u] = __ballot_sync(0xffffffffu, on);
          const int sv = v >> lognblk;
          if (sv < m) {
            const int tv = tg + sv < C::kTags ? tg + sv : tg + sv - C::kTags;
            c.tag[tv].at[v & (nblk - 1)] =
                on ? ent * block_bytes + (long long)w.h * head_bytes +
                         (long long)(((w.k + sv) * kKeys) & (B - 1)) * row_bytes
                   : -1ll;
          }
        }
        const int n = w.k1 - w.k0, i = w.k - w.k0 + k;   // stages of the part, this lane's
        if (w.k == w.k0) {   // the part begins
          const long long w2 = 2 * a.BM;
          const int left = (int)min((long long)w.L - w2 * w.pr, w2);   // the pair's tokens
          const int ntok_a = min(left, a.BM), ntok_b = left - ntok_a;
          const int nkt = w.nkt(), klo = w.lo / kKeys;
          const int p0 = w.T - w.L + (int)(w2 * w.pr);
          nkt_a = ntok_b == 0 ? nkt : (p0 + ntok_a - 1) / kKeys + 1;
          part = (ntok_b == 0 ? kAlt | (n >= 2 ? kHasB : 0) : 0) | (w.k0 == klo ? kBegins : 0) |
                 (w.k0 == klo && w.k1 >= nkt_a ? kWholeA : 0) |
                 (w.k0 == klo && w.k1 == nkt ? kWholeB : 0);
          if (lane < min(m, 2)) {   // tile B's first stage may be the second
            t.part = parts;
            t.h = w.h;
            t.q0 = w.q0 + (int)(w2 * w.pr);
            t.p0 = p0;
            t.lo = w.lo;
            t.ntok_a = ntok_a;
            t.ntok_b = ntok_b;
            t.nkt_a = nkt_a;
            t.nkt = nkt;
            t.i0 = w.i0;
            t.len = w.length(a);
          }
          ++parts;
        }
        const int kt = w.k + k;
        int f = part | (i == 0 ? kFirst | kFirstA : 0) | (i == n - 1 ? kLast : 0);
        if (part & kAlt) {
          f |= (i & 1) ? kActB : kActA;
          if (i == 1) f |= kFirstB;
          if (i + 2 >= n) f |= (i & 1) ? kLastB : kLastA;
        } else {
          f |= kActB | (kt < nkt_a ? kActA : 0) | (i == 0 ? kFirstB : 0) |
               (i == n - 1 ? kLastB : 0) | (kt == min(w.k1, nkt_a) - 1 ? kLastA : 0);
        }
        // the pieces of this lane's stage that are to be read, and that are there
        const int v0 = k << lognblk;
        uint32_t mine = got[0], wanted = want[0];
#pragma unroll
        for (int u = 1; u < kRounds; ++u)
          if ((v0 >> 5) == u) {
            mine = got[u];
            wanted = want[u];
          }
        const uint32_t all = 0xffffffffu >> (32 - nblk);
        mine = (mine >> (v0 & 31)) & all;
        wanted = (wanted >> (v0 & 31)) & all;
        uint4 mask = make_uint4(0u, 0u, 0u, 0u);
        const int live = w.end - kt * kKeys;   // keys before the pair's end
        if (live < kKeys || mine != all) {
          // rows that hold data, and rows of blocks that are out of range
          uint64_t rows = 0ull, bad = 0ull;
          for (int b = 0; b < nblk; ++b) {
            const uint64_t bits = (~0ull >> (64 - bs)) << (b * bs);
            if ((mine >> b) & 1u) rows |= bits;
            else if ((wanted >> b) & 1u) bad |= bits;
          }
          if (live < kKeys) {
            rows &= (1ull << live) - 1ull;
            bad &= (1ull << live) - 1ull;
          }
          f |= kEdge | (bad ? kMarked : 0);
          mask.x = (uint32_t)bad;
          mask.y = (uint32_t)(bad >> 32);
          if (lane < m) {
            t.rows[0] = (uint32_t)rows;
            t.rows[1] = (uint32_t)(rows >> 32);
          }
        }
        if (lane < m) {
          *reinterpret_cast<uint4*>(t.mask) = mask;
          t.flags = f;
          t.kt = kt;
        }
        __syncwarp();
        if (lane < m) mbar_arrive(smem_u32(&c.tfull[bk]));
        w.k += m;
        ts += m;
        if (ts >= C::kAhead) {
          ts -= C::kAhead;
          ph ^= 1u;
        }
        tg += m;
        if (tg >= C::kTags) tg -= C::kTags;
      }
    }
    __syncwarp();
  } else if (warp >= kConvert) {
    setmaxnreg_dec<kRegsConvert>();
    // ========================= conversion =========================
    const int x = tid & 127;                        // thread of the warpgroup
    const int w = warp & 3;                         // rows 16 w .. of a stage
    const int kv = (warp - kConvert) >> 2;          // K or V, tile A's queries or B's
    const uint32_t inv_g = (65535u + (uint32_t)a.G) / (uint32_t)a.G;   // row / G, row < 128
    const int B = 1 << a.log2B, log2s = min(a.log2B, 6);
    // A lane's pieces: 16 bytes of kRows rows, as words (8 codes of 4 bits) or
    // double words (8 codes of 8 bits), each of which becomes one 16-byte chunk of
    // the swizzled operand.  A lane takes word j ^ turn as its j-th: `turn` is such
    // that neither the loads of a warp nor the stores of eight neighbours meet in
    // a bank (rows lie kRowBytes apart in the ring, and chunk k of an operand's row
    // r at k ^ r % 8).
    constexpr int kPieces = kFour ? D / 32 : D / 16;   // of a row
    constexpr int kRowsStep = 32 / kPieces;            // rows of a warp's load
    constexpr int kRows = 16 / kRowsStep;
    constexpr int kWords = kFour ? 4 : 2;
    const int col = lane % kPieces, rl = lane / kPieces;
    const int turn = kFour ? (D == 128 ? (((col >> 1) << 1) ^ (rl & 1) ^ (rl & 3) ^ ((rl >> 2) & 1))
                                       : ((rl >> 2) & 3))
                           : (D == 128 ? ((col >> 2) ^ (rl & 1)) : ((rl >> 1) & 1));
    const uint32_t mine = ring + (uint32_t)((4 * kv + w) * R::kWarp);
    const uint32_t from = mine + (uint32_t)(rl * R::kRowBytes + 16 * col + (16 / kWords) * turn);
    const uint32_t scales = mine + (uint32_t)(R::kCodes + (rl >> 2) * (D / 4) + 8 * col);
    // the copies: this lane's bytes of its rows, behind the piece they lie in
    const uint8_t* const pool = kv ? a.vc : a.kc;
    const int row_bytes = kFour ? D / 2 : a.H * D;   // (a block's bytes fit in 31 bits)
    int piece[kRows], sc_piece = 0, src[kRows], sc_src = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = 16 * w + rl + kRowsStep * i;
      piece[i] = row >> log2s;
      src[i] = (row & ((1 << log2s) - 1)) * row_bytes + 16 * col;
    }
    constexpr int kScalePieces = kFour ? D / 16 : 0;   // 16 bytes each
    if constexpr (kFour) {
      const int q = lane / (D / 64), row = 16 * w + 4 * q;
      sc_piece = (row & 63) >> log2s;
      sc_src = B * (D / 2) + (row & ((1 << log2s) - 1)) * (D / 16) + 16 * (lane % (D / 64));
    }
    // Fetching a stage: its tag is looked at, on the chance that it is written, before
    // the conversion of another, whose time hides the look; the copies are issued
    // behind it.  The tag is read behind a branch on the test.  A form that read it beside
    // the test, in program order behind it, and used it where the test had passed got, in
    // one of some 10^4 calls, what the place had held before; neither the program's order
    // nor the memory model explains that, and the cause is not known.
    long long at[kRows], sc_at = -1;
    int next_rs = 0, next_ts = 0, next_tg = 0;    // of the stage to be fetched next
    int next_flags = 0;
    uint32_t next_ph = 0u;
    bool ok = true, more = true, written = false;
    auto read_tag = [&]() {
      const Tag& t = c.tag[next_tg];
      next_flags = t.flags;
#pragma unroll
      for (int i = 0; i < kRows; ++i) at[i] = t.at[piece[i]];
      if constexpr (kFour) {
        // `at` counts a larger block's rows before the piece by their codes
        const int r = (t.kt * kKeys) & (B - 1) & ~(kKeys - 1);
        sc_at = t.at[sc_piece];
        if (sc_at >= 0) sc_at += sc_src - r * (D / 2 - D / 16);
        if (lane >= kScalePieces) sc_at = -1;
      }
    };
    auto look = [&]() {
      written = __all_sync(0xffffffffu, mbar_test(smem_u32(&c.tfull[next_ts]), next_ph)) != 0;
      if (written) read_tag();
    };
    auto fetch = [&]() {
      if (more) {
        if (!written) {
          ok = ok && wait_warp(c.tfull[next_ts], next_ph);
          read_tag();
        }
        more = ok && !(next_flags & kStop);
      }
      if (more) {
        const uint32_t slot = (uint32_t)(next_rs * R::kStage);
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          if (at[i] >= 0)
            copy16(mine + slot + (uint32_t)((rl + kRowsStep * i) * R::kRowBytes + 16 * col),
                   pool + (at[i] + src[i]));
        if constexpr (kFour)
          if (sc_at >= 0) copy16(mine + slot + (uint32_t)(R::kCodes + 16 * lane), pool + sc_at);
        if (++next_rs == R::kRing) next_rs = 0;
        if (++next_ts == C::kAhead) {
          next_ts = 0;
          next_ph ^= 1u;
        }
        if (++next_tg == C::kTags) next_tg = 0;
      }
      commit_copies();   // a group a stage, fetched or not
    };
    uint32_t chunk[kWords];
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      const int k = kWords * col + (j ^ turn);   // 8 columns of the row
      chunk[j] = stages + (uint32_t)(k >> 3) * X::kPlane + (uint32_t)(16 * w + rl) * 128u +
                 (uint32_t)((k ^ rl) & 7) * 16u;
    }
    // the two scale bytes of a row's piece, the first for the lane's first words
    const uint32_t pick = (uint32_t)(((turn & 2) ? 0x04 : 0x40) + 0x11 * (rl & 3));
    int st = 0, rs = 0, ts = 0, tg = 0;           // slots: operands, codes, barriers, tags
    uint32_t ph = 0u;
#pragma unroll 1
    for (int k = 0; k < R::kRing; ++k) {
      written = false;
      fetch();
    }
    int flags = ok ? c.tag[0].flags : 0;
    bool free = false;   // the stage's operands, tried ahead
    while (ok) {
      if (!__all_sync(0xffffffffu, free) && !wait_warp(c.empty[st], ph ^ 1u)) {
        ok = false;
        break;
      }
      Tag& t = c.tag[tg];
      if (flags & kStop) {   // the tag that ended the fetches
        warp_arrive(c.full[st]);
        break;
      }
      if (flags & kFirst) {
        if (!wait_warp(c.qempty, ((uint32_t)t.part & 1u) ^ 1u)) {
          ok = false;
          break;
        }
        // ---- a warp's 32 query rows of a tile, a few whole rows a copy
        if (kv == 0 || t.ntok_b > 0) {
          const uint32_t qt = qtiles + (uint32_t)kv * X::kQTile;
          const int rows = (kv ? t.ntok_b : t.ntok_a) * a.G;
          constexpr int kChunks = D / 8, kStep = 32 / kChunks;   // of 16 bytes; rows a copy
          const int qc = lane % kChunks;
          const uint16_t* const src =
              a.q + ((size_t)(t.q0 + kv * a.BM) * a.Hq + (size_t)t.h * a.G) * D + 8 * qc;
#pragma unroll 2
          for (int i = 0; i < 32; i += kStep) {
            const int row = 32 * w + i + lane / kChunks;
            const uint32_t dst = qt + (uint32_t)(qc >> 3) * X::kQPlane + (uint32_t)row * 128u +
                                 (uint32_t)((qc ^ row) & 7) * 16u;
            const int tok = (int)((uint32_t)row * inv_g >> 16);
            if (row < rows)
              copy16(dst, reinterpret_cast<const uint8_t*>(
                              src + ((size_t)tok * (a.Hq - a.G) + row) * D));
            else sts16(dst, 0u, 0u, 0u, 0u);
          }
          commit_copies();
          wait_copies<0>();
          __syncwarp();
          float back = 1.f;
          if constexpr (kBF16) {
            // A bfloat16 row is brought into binary16's range, where it lies, by a
            // power of two (its largest magnitude into [1, 2)), which its score
            // factor takes back; elements 2^-14 below the largest lose bits below
            // 2^-24 of it.  Thread x holds row x.
            const uint32_t at = qt + (uint32_t)x * 128u;
            float mx = 0.f;
#pragma unroll 4
            for (int j = 0; j < D / 8; ++j) {
              const uint4 y = lds16(at + (uint32_t)(j >> 3) * X::kQPlane +
                                    (uint32_t)((j ^ x) & 7) * 16u);
              const uint32_t z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = unpack2<true>(z[e]);
                mx = max3f(mx, fabsf(f.x), fabsf(f.y));
              }
            }
            // 2^e <= mx < 2^(e+1); zero, subnormal or infinite maxima keep a
            // factor whose inverse is a normal number
            const int e = min(max((int)(__float_as_uint(mx) >> 23), 1), 253);
            back = __uint_as_float((uint32_t)e << 23);
            const float to = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll 4
            for (int j = 0; j < D / 8; ++j) {
              const uint32_t p = at + (uint32_t)(j >> 3) * X::kQPlane +
                                 (uint32_t)((j ^ x) & 7) * 16u;
              const uint4 y = lds16(p);
              uint32_t z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = unpack2<true>(z[e]);
                z[e] = pack2<false>(f.x * to, f.y * to);
              }
              sts16(p, z[0], z[1], z[2], z[3]);
            }
          }
          c.factor[t.part % (S + 1)][kv][x] = a.scale_log2 * back;
        }
      }
      // ---- the stage's keys or values to 16 bits
      look();
      const int tg1 = tg + 1 == C::kTags ? 0 : tg + 1;
      const int flags1 = c.tag[tg1].flags;   // of the stage after this one
      wait_copies<R::kRing - 1>();
      __syncwarp();   // every lane's copies have landed
      const uint32_t f0 = from + (uint32_t)(rs * R::kStage);
      const uint32_t to = (uint32_t)st * X::kStage + (uint32_t)kv * X::kPart;
      uint32_t y[kRows][4], sc[kRows], odd = 0u;   // odd: bytes that are NaN
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if constexpr (kFour) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            y[i][j] = lds4((f0 ^ (uint32_t)(4 * j)) + (uint32_t)(kRowsStep * i * R::kRowBytes));
          const uint2 s2 = lds8(scales + (uint32_t)(rs * R::kStage) +
                                (uint32_t)(kRowsStep * i / 4 * (D / 4)));
          sc[i] = prmt(s2.x, s2.y, pick) & 0xffffu;
          if (kv) odd |= nan_bytes(sc[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint2 z = lds8((f0 ^ (uint32_t)(8 * j)) + (uint32_t)(kRowsStep * i * R::kRowBytes));
            y[i][2 * j] = z.x;
            y[i][2 * j + 1] = z.y;
          }
          if (kv) odd |= nan_bytes(y[i][0]) | nan_bytes(y[i][1]) | nan_bytes(y[i][2]) |
                         nan_bytes(y[i][3]);
        }
      }
      if ((flags & kEdge) || __any_sync(0xffffffffu, odd != 0u)) {
        // rows that hold no data, and NaN among the values, become zeros: a weight
        // of zero times NaN would reach rows that do not attend to them
        const uint32_t live = (flags & kEdge) ? t.rows[w >> 1] >> (16 * (w & 1)) : 0xffffu;
        uint32_t nan = 0u;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int rr = rl + kRowsStep * i;   // of the warp's rows
          const bool in = ((live >> rr) & 1u) != 0u;
          uint32_t bad = 0u;
          if (kv)
            bad = kFour ? nan_bytes(sc[i])
                        : nan_bytes(y[i][0]) | nan_bytes(y[i][1]) | nan_bytes(y[i][2]) |
                              nan_bytes(y[i][3]);
          if (in && bad) nan |= 1u << rr;
          if (!in || bad) sc[i] = y[i][0] = y[i][1] = y[i][2] = y[i][3] = 0u;
        }
        nan = __reduce_or_sync(0xffffffffu, nan);
        if (nan && lane == 0) {
          atomicOr(&t.mask[2 + (w >> 1)], nan << (16 * (w & 1)));
          atomicOr(&t.flags, kMarked);
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        // rows 4 apart swap halves of the swizzle
        const uint32_t flip = (kRowsStep * i) & 4 ? 64u : 0u;
        uint32_t s = 0u;
        if constexpr (kFour) s = e4m3x2_to_f16x2(sc[i]);
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          uint32_t f[4];
          if constexpr (kFour) {
            e2m1x8_to_f16x2(y[i][j], f);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = j < 2 ? hmul2_lo(f[e], s) : hmul2_hi(f[e], s);
          } else {
            e4m3x4_to_f16x2x2(y[i][2 * j], f[0], f[1]);
            e4m3x4_to_f16x2x2(y[i][2 * j + 1], f[2], f[3]);
          }
          sts16((chunk[j] ^ flip) + to + (uint32_t)(kRowsStep * i * 128), f[0], f[1], f[2], f[3]);
        }
      }
      fence_proxy_async_smem();   // the operands, before the tensor core reads them
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&c.full[st]));
        mbar_arrive(smem_u32(&c.tempty[ts]));
      }
      fetch();   // into the ring's place that is free now
      if (++rs == R::kRing) rs = 0;
      if (++ts == C::kAhead) ts = 0;
      if (++st == S) {
        st = 0;
        ph ^= 1u;
      }
      tg = tg1;
      flags = flags1;
      free = mbar_test(smem_u32(&c.empty[st]), ph ^ 1u);
    }
    if (!ok && lane == 0) give_up();
    wait_copies<0>();   // nothing lands in shared memory after the block's end
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ========================= softmax =========================
    const int tile = warp >> 2, wq = warp & 3;
    const int r = tid & 127;
    const uint32_t trow = tmem + ((uint32_t)(32 * wq) << 16);
    const uint32_t tcol = trow + (uint32_t)(256 * tile);
    unsigned long long* const tb = c.tile[tile];
    const int firstbit = tile ? kFirstB : kFirstA, lastbit = tile ? kLastB : kLastA;
    const int tok_r = r / a.G;
    int ntok = 0, p0 = 0, prow = -1;
    bool busy = false;             // some row of this warp is a row
    int h = 0, q0 = 0, lo = 0, nkt_t = 0;   // of the part
    long long i0 = 0, line = 0;
    float factor = 0.f, m_used = -INFINITY, l = 0.f;
    bool poison = false;
    bool ok = true;
    int nt = 0, nb_alt = 0, nm = 0;   // scores read, pairs in turn joined, meetings
    // The tile's four warps wait for one another, with a limit: a warp whose wait ran out
    // has left, and one that looked at the same barrier a moment later has not (a named
    // barrier would hold it for good).
    auto meet = [&]() {
      warp_arrive(c.met[tile]);
      return wait_warp(c.met[tile], (uint32_t)nm++ & 1u);
    };
    while (true) {
      if (!wait_warp(tb[kSFull], (uint32_t)nt & 1u)) {
        ok = false;
        break;
      }
      const int4 rec = c.scores[tile][nt & 3];
      const int flags = rec.x, kt = rec.y;
      if (flags & kStop) break;
      uint4 mk = make_uint4(0u, 0u, 0u, 0u);
      if (flags & (firstbit | kMarked)) {
        const Tag& tg = c.tag[rec.w];
        mk = *reinterpret_cast<const uint4*>(tg.mask);
        if (flags & firstbit) {
          h = tg.h;
          q0 = tg.q0;
          lo = tg.lo;
          nkt_t = tile ? tg.nkt : tg.nkt_a;
          i0 = tg.i0;
          line = tg.len;
          const bool other = tile == 1 && !(flags & kAlt);   // rows of the second tile
          ntok = other ? tg.ntok_b : tg.ntok_a;
          p0 = tg.p0 + (other ? a.BM : 0);
          const bool valid = r < a.BM * a.G && tok_r < ntok;
          prow = valid ? p0 + tok_r : -1;
          busy = 32 * wq < ntok * a.G;
          factor = c.factor[tg.part % (S + 1)][other ? 1 : 0][r];
          m_used = -INFINITY;
          l = 0.f;
          poison = false;
        }
      }
      warp_arrive(c.empty[rec.z]);   // the tag is read
      if (busy) {
        tc_fence_after();
        uint32_t sr[kKeys];
        tmem_ld32(tcol, *reinterpret_cast<uint32_t(*)[32]>(sr));
        tmem_ld32(tcol + 32, *reinterpret_cast<uint32_t(*)[32]>(sr + 32));
        tmem_wait_ld();
        tc_fence_before();
        warp_arrive(tb[kSFree]);
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
        const bool plain = t0 + (kKeys - 1) <= p0 && (flags & kMarked) == 0 &&
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
        warp_arrive(tb[kSFree]);
      }
      warp_arrive(tb[kPFull + (nt & 1)]);
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
          warp_arrive(c.bdone);
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
                  *reinterpret_cast<uint4*>(rec + 4 * ((cc / 4 + e) * kTileRows + r)) =
                      make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
              }
              __syncwarp();
            }
          }
          tc_fence_before();
          warp_arrive(tb[kOFree]);
          if (join) warp_arrive(c.tile[1][kOFree]);
          if (!whole) {
            if (prow >= 0) {
              rec[(size_t)kTileRows * D + r] = m_used;
              rec[(size_t)kTileRows * (D + 1) + r] = l;
            }
            if (!meet()) {
              ok = false;
              break;
            }
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
                  const int s0 = stage_at(c.bound[b] - i0, lo, nkt_t, a.start);
                  in = s0 < stage_at(c.bound[b + 1] - i0, lo, nkt_t, a.start);
                  begins = s0 == lo / kKeys;
                }
                const uint32_t all = __ballot_sync(0xffffffffu, in);
                if (in) c.parts[tile][n + __popc(all & ((1u << lane) - 1u))] =
                    (uint16_t)(b * 2 + (begins ? 1 : 0));
                n += __popc(all);
                if (all) end = b0 + 31 - __clz(all);
              }
              if (lane == 0) {
                c.nparts[tile] = n;
                // releases this tile's record (ordered before by the meeting),
                // acquires those counted before it
                uint32_t* const cnt = a.ws_count + 2 * end + tile;
                const bool last = atom_add_acq_rel_gpu(cnt, 1u) + 1u == (uint32_t)n;
                if (last) *cnt = 0u;   // ready for the next call
                c.last[tile] = last ? 1 : 0;
              }
            }
            if (!meet()) {
              ok = false;
              break;
            }
            if (c.last[tile]) {
              // ---- the last record: join them all, in the order of the keys.  A
              // thread finds its row's maximum and sum, then takes vectors of rows: a
              // warp four neighbouring ones of eight rows
              constexpr int kAhead = 4, kHalves = D / 64;
              const int n = c.nparts[tile], rows = ntok * a.G;
              const float* const recs = a.ws_rec + (size_t)tile * rec_floats(D);
              auto record = [&](int k) {
                return recs + (size_t)c.parts[tile][k] * 2 * rec_floats(D);
              };
              if (r < rows) {
                float m = -INFINITY, ls = 0.f;
                for (int k = 0; k < n; ++k) {
                  const float* const p = record(k) + (size_t)kTileRows * D + r;
                  const float pm = __ldcg(p), pl = __ldcg(p + kTileRows);
                  const float mn = fmaxf(m, pm), base = mn == -INFINITY ? 0.f : mn;
                  ls = ls * ex2_approx(m - base) + pl * ex2_approx(pm - base);
                  m = mn;
                }
                c.join[tile][r][0] = m == -INFINITY ? 0.f : m;
                c.join[tile][r][1] = ls == 0.f ? 0.f : a.v_scale / ls;
              }
              if (!meet()) {
                ok = false;
                break;
              }
              for (int u = 0; u < (rows + 31) / 32 * kHalves; ++u) {
                const int r0 = 32 * (u / kHalves) + (lane & 7);
                const int vec = 16 * (u % kHalves) + 4 * wq + (lane >> 3), col = 4 * vec;
                float4 acc[kAhead];
#pragma unroll
                for (int b = 0; b < kAhead; ++b) acc[b] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < n; ++k) {
                  const float* const p = record(k);
                  float4 v[kAhead];
                  float w[kAhead];
#pragma unroll
                  for (int b = 0; b < kAhead; ++b) {
                    const int rr = min(r0 + 8 * b, rows - 1);
                    v[b] = __ldcg(reinterpret_cast<const float4*>(p + 4 * (vec * kTileRows + rr)));
                    w[b] = __ldcg(p + (size_t)kTileRows * D + rr);
                  }
#pragma unroll
                  for (int b = 0; b < kAhead; ++b) {
                    const int rr = min(r0 + 8 * b, rows - 1);
                    const float f = ex2_approx(w[b] - c.join[tile][rr][0]);
                    acc[b].x = fmaf(v[b].x, f, acc[b].x);
                    acc[b].y = fmaf(v[b].y, f, acc[b].y);
                    acc[b].z = fmaf(v[b].z, f, acc[b].z);
                    acc[b].w = fmaf(v[b].w, f, acc[b].w);
                  }
                }
#pragma unroll
                for (int b = 0; b < kAhead; ++b) {
                  const int rr = r0 + 8 * b;
                  if (rr >= rows) break;
                  const float mul = c.join[tile][rr][1];
                  const int tok = rr / a.G;
                  uint16_t* const dst =
                      a.out + ((size_t)(q0 + (tile ? a.BM : 0) + tok) * a.Hq + (size_t)h * a.G +
                               (rr - tok * a.G)) * D + col;
                  *reinterpret_cast<uint2*>(dst) =
                      make_uint2(pack2<kBF16>(acc[b].x * mul, acc[b].y * mul),
                                 pack2<kBF16>(acc[b].z * mul, acc[b].w * mul));
                }
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
  if (warp == kTagger) tmem_dealloc(tmem, 512);
}

}  // namespace

}  // namespace pa

#include "pa_prefill_few.cuh"

namespace pa {

namespace {

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

// The workspace: counters of this kernel, then of the other; records of this one,
// four a block, then of the other, two a block.
constexpr size_t kFewCounters = PA_PREFILL_QUANT_COUNTERS / 2;
inline size_t few_records_at(int D, int grid) {
  return PA_PREFILL_QUANT_COUNTERS + (size_t)grid * 4 * rec_floats(D) * sizeof(float);
}
inline size_t prefill_quant_bytes(int D, int grid) {
  return few_records_at(D, grid) +
         (size_t)kFewBlocks * grid * 2 * few_rec_floats(D) * sizeof(float);
}
static_assert(2 * kMaxGrid * sizeof(uint32_t) <= kFewCounters &&
                  kFewBlocks * kMaxGrid * sizeof(uint32_t) <= PA_PREFILL_QUANT_COUNTERS - kFewCounters,
              "a block's counters");

// Average rows a sequence up to which a batch is split between the two kernels (the
// lengths themselves are on the device).
constexpr int kFewAverage = 192;

// The kernels' opt-in to their shared memory, once a device.
constexpr int kMaxDevices = 64;

template <int D, bool kBF16, bool kFour>
int launch_prefill_quant(const Args& a, int grid, int device, cudaStream_t s) {
  static std::mutex mu;
  static bool ready[kMaxDevices];
  const auto kern = prefill_quant_kernel<D, kBF16, kFour>;
  const auto few = prefill_few_kernel<D, kBF16, kFour>;
  constexpr size_t smem = smem_bytes<D, kFour>(), few_smem = sizeof(FewShared<D, kFour>);
  static_assert(smem <= 227 * 1024 && kFewBlocks * few_smem <= 224 * 1024, "a block's shared memory");
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[device]) {
      cudaError_t e =
          cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      cudaFuncAttributes at{};
      if (!e) e = cudaFuncGetAttributes(&at, kern);
      if (e) return launch_status(e, "cudaFuncSetAttribute (quantized prefill)");
      // the roles re-divide the launch's registers, which the increases wait for
      if (at.numRegs != kRegsLaunch) return PA_ERR_UNSUPPORTED;
      e = cudaFuncSetAttribute(few, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)few_smem);
      if (e) return launch_status(e, "cudaFuncSetAttribute (quantized prefill of few rows)");
      ready[device] = true;
    }
  }
  clear_stale_error();
  if (a.few != kFewOnly)
    if (int rc = launch_status(launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads), smem, s, a),
                               "quantized prefill launch"))
      return rc;
  if (a.few == kFewNone) return PA_OK;
  return launch_status(launch_pdl(few, dim3((unsigned)(kFewBlocks * grid)), dim3(kFewThreads), few_smem, s, a),
                       "quantized prefill launch (few rows)");
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
  a.start = kStart[q_dtype == PA_BF16 ? 1 : 0];
  // Sequences of few rows have a kernel of their own.  If even all of total_q in one
  // would be one, it is the only one; both run where the average of the sequences is not
  // far beyond.  An average cannot tell who they are: a few long chunks hide single
  // tokens, and chunks that are all of some 30 rows pay for a launch that finds nothing.
  // Us with the kernel of 128-row tiles alone / with both: 64 single tokens over 2 to 8 K
  // of 4 bits beside a chunk of 512 425 / 241 (both run); 63 beside a chunk of 2,048 288 /
  // 265, 64 beside one of 8,192 3,242 / 3,130, 64 beside four of 2,048 730 / 676 (tiles
  // alone); 32 verified proposals of 4 tokens over 2 to 4 K 101 / 111 (both); 16 chunks of
  // 512 550 / 568, one of 64 tokens 14.9 / 17.4 (tiles alone).
  const long long rows = (long long)total_q * a.G;
  a.few = rows <= kFewRows ? kFewOnly
                           : (rows <= (long long)kFewAverage * num_seqs ? kFewBoth : kFewNone);
  a.few_count = a.ws_count + kFewCounters / sizeof(uint32_t);
  a.few_rec = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                       few_records_at(head_dim, grid));
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
