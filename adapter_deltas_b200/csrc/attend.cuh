// attend.cuh -- attention of one new token per sequence over the paged cache.
//
// For query head h of sequence s, with key head g = h / (n_heads / heads) and
// positions j in [max(0, len - window), len):
//     s_j = scale * q . k_j,   out = sum_j e^(s_j) v_j / (sum_j e^(s_j) + e^sink),
// in one pass over the cache with a running maximum m and sum l: a step of
// tokens gives m' = max(m, max s_j), l' = l e^(m - m') + sum e^(s_j - m'), and the
// weighted values are rescaled by e^(m - m') when the maximum moved (in base
// 2 throughout: log2(e) is folded into the scale).  Two such states over
// disjoint tokens join by the same formula, so the tokens can be cut anywhere.
//
// Bound by HBM: 4 flops per cached element and query head, at most 16 query
// heads to a byte.  (64 requests of 200 to 4000 tokens, bf16, 32 heads of 128: 1.15 GB
// in 182 us, 6.3 TB/s; 512 of 64 to 2048, e4m3, 32 / 8 heads: 585 MB in 111 us, 5.3 TB/s.
// Short calls are latency: 16 requests of up to 100 tokens 9 us.)  So the split is by bytes, evenly, whatever the lengths:
//  - The batch is one flat list of slots, ordered by (sequence, unit, step).  A
//    unit is one key head with up to 8 (or 16) of its query heads; a step is 16
//    TT consecutive tokens of it.  A unit has one slot for each step and one
//    before them for what it costs to begin and end one (about a step's time).
//    Each block takes an equal range of the list (one block per SM), each of its
//    warps an equal range of the block's.  Every block finds its place itself from
//    the lengths (one scan), so there is no plan to keep and nothing of it is read
//    on the host.
//  - A warp is on its own: one lane fetches its steps' tiles with bulk copies
//    (one per 16 tokens: a tile is contiguous in the cache, K, V and scales)
//    into the warp's ring of stages, several steps ahead, through the page
//    table; there is no block-wide synchronisation until the end.
//  - A (sequence, unit) that lies inside one warp's range is written at once.
//    States of ranges that cut one are joined in the block, in token order;
//    what a block's border cuts goes to the workspace, and the last of a unit's
//    blocks to get there joins them (in order again, whichever block it is:
//    equal inputs give equal bits).  Blocks count themselves in, none waits for
//    another.  (As a second launch the join took 4 to 6 us.)
//
// The products run on the warp-level tensor instruction (m16n8k16): a unit's 8
// query heads are the N = 8 of both products, S^T = K q^T (16 tokens x 8 heads)
// and O^T += V^T P^T (16 dims x 8 heads), K and V read from the staged tile as the
// A operand.  (With the heads as M half of each instruction and of the
// accumulators would be padding; tcgen05 takes no fewer than 64 rows.)  The
// weights leave S^T token by token and are needed head by head: one movmatrix
// per 8 x 8 block turns them.  8-bit codes become
// fp16 exactly, in 2 to 5 instructions per four; K's scales multiply the
// scores, V's the weights, in fp32.
//
// More than 16 query heads to a key head are several units, each of which reads
// the key head's tiles again (128 requests of 2000 to 4000 tokens over one key head
// of 128, bf16: 45 us for 16 heads, 61 for 32, 101 for 64).
//
// Tokens outside the range get weight 0 by selection, not by adding: what lies
// in their places (the end of a page, before the window) may be anything.
#pragma once

#include <cfloat>

#include "kv.cuh"

namespace lora {

constexpr int kAttMaxWarps = 12;
constexpr int kAttMaxStages = 8;
constexpr int kAttSmem = 227 * 1024;
constexpr int kSlack = 4, kWeight = 11;  // powers of two (kWeight + kSlack: within fp16)
constexpr int kCutSteps = 3;  // 3 to 12 choose alike in all that was measured
constexpr int kMaxSlotsLog2 = 30;  // of a block: counted in 32 bits

struct AttendArgs {
  const uint8_t *q;
  uint8_t *out;
  long long ldq, ldo;  // bytes
  float *lse;
  const float *sinks;
  int n_heads, group;  // query heads, and of them per key head
  int units;           // per sequence: heads * head groups
  int head_groups;
  int rows;            // of a state: query heads of a unit (the last unit of a key head may have fewer)
  float scale2;        // scale * log2(e)
  int window;
  int n_stages;
  int stall;           // test only: kStallAll, or kStallLane + a lane
  unsigned long long wait_ns;
  // workspace: what each block's borders cut
  unsigned long long *done;  // [blocks] how many blocks of the unit that starts in a block and goes on are done
  unsigned long long tag;    // of this launch, in done's upper bits: whatever is there from before counts as none
  float *part;         // [blocks][2] states: 0 continues from the block before, 1 starts here
  float *first;        // [blocks][warps] states: a warp's first piece, when more of its range follows,
  int first_in_smem;   // or where in shared memory those are (0: not there)
};

constexpr int kCountBits = 16;  // of done

// A state in memory: m[rows], l[rows] (each row's place a multiple of 16 bytes
// from the start: rows * 2 rounded up to 4 floats), then rows x dim weighted sums.
__host__ __device__ constexpr int state_head(int rows) { return (2 * rows + 3) & ~3; }
__host__ __device__ constexpr int state_floats(int rows, int dim) { return state_head(rows) + rows * dim; }

// ------------------------------------------------------------------ pieces

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// 8 x 8 of 16-bit values, transposed: a thread has two neighbours of a row.
__device__ __forceinline__ uint32_t turn(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float log2_fast(float x) {  // (0: minus infinity)
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Bytes 0 and 2 (even) and 1 and 3 (odd) of a word of codes as fp16 pairs, exactly.
//  int8: 1024 + (code + 128) is fp16 with the code's bits in its low byte.
template <int TYPE>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &even, uint32_t &odd) {
  if (TYPE == LORA_KV_E4M3) {
    const uint32_t x = __byte_perm(w, 0, 0x3120);
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(even), "=r"(odd)
        : "r"(x));
  } else {
    const uint32_t x = w ^ 0x80808080u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(even) : "r"(__byte_perm(x, 0x64646464u, 0x4240)), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(odd) : "r"(__byte_perm(x, 0x64646464u, 0x4341)), "r"(0x64806480u));
  }
}

// A word of K codes as two fp16 pairs: e4m3 bytes 0, 1 and 2, 3 (one instruction
// each); int8 bytes 0, 2 and 1, 3.
template <int TYPE>
__device__ __forceinline__ void key_codes_to_f16(uint32_t w, uint32_t &a, uint32_t &b) {
  if (TYPE == LORA_KV_E4M3)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(w));
  else
    codes_to_f16<TYPE>(w, a, b);
}

// The same word of K codes as two bf16 pairs, exactly: e4m3 codes times 2^-120 (their
// bits in bf16's place: its exponents start that much lower); int8 as the
// difference of 128 + the code's low bits and 128 or, where it is negative, 256.
constexpr float kFineScale = 0x1p120f;
template <int TYPE>
__device__ __forceinline__ void key_codes_to_bf16(uint32_t w, uint32_t &a, uint32_t &b) {
  if (TYPE == LORA_KV_E4M3) {
    const uint32_t x = __byte_perm(w, 0, 0x1404), y = __byte_perm(w, 0, 0x3424);
    a = (x & 0x80008000u) | (x >> 4 & 0x07f007f0u);
    b = (y & 0x80008000u) | (y >> 4 & 0x07f007f0u);
  } else {
    const uint32_t x = __byte_perm(w, 0x43434343u, 0x4240), y = __byte_perm(w, 0x43434343u, 0x4341);
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(x & 0xff7fff7fu), "r"(x & 0xff80ff80u));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(y & 0xff7fff7fu), "r"(y & 0xff80ff80u));
  }
}

// Over a bf16 cache scores are q as it is times the keys.  Over an 8-bit cache keys
// become fp16 exactly, and q is scaled per head by a power of two to below 2^16: fp16
// then has all bits of what is 2^-kFine of the head's largest |q| or more.  A unit with
// a smaller q is multiplied in bf16 instead, which has all of q and of the codes too
// but takes more instructions to make.  (As three int8 terms times int8 codes, 2^-22
// of the largest |q| was lost and 256 requests of 2000 int8 tokens took 105.5 us
// instead of 103.9; the warp-level product of e4m3 operands is no single instruction
// of this GPU and took 1.7 times the instructions.)
constexpr float kQTop = 0x1p15f;
constexpr int kFine = 32;

// A length that is attended to, else 0 (none, empty, in error).
__device__ __forceinline__ int valid_len(const KvView &kv, const KvSeqs &s, int len) {
  return len > 0 && kv_len_ok(kv, s, len) ? len : 0;
}
__device__ __forceinline__ int seq_len(const KvView &kv, const KvSeqs &s, int i) {
  return valid_len(kv, s, __ldg(s.lens + i));
}
__device__ __forceinline__ int first_token(int len, int window) { return window && len > window ? len - window : 0; }
// Slots of a unit of a sequence: one, and one for each step of tt tiles (aligned
// to that) from the first token's to the last one's.  None without a token.
__device__ __forceinline__ int unit_slots(int len, int window, int tt) {
  const int per = kTileTokens * tt;
  return len ? (len + per - 1) / per - first_token(len, window) / per + 1 : 0;
}

// Write row r's result from its state: o = sums for 4 dims, m and l over all tokens.
struct Ends {
  float mul, lse;
};
__device__ __forceinline__ Ends finish(const float *sinks, int head, float m, float l) {
  Ends e;
  const float given = sinks ? sinks[head] : -INFINITY;
  // (in base 2 within the range too: one at its end is a number still)
  const float sink = fabsf(given) < INFINITY ? fminf(fmaxf(given * 1.44269504f, -FLT_MAX), FLT_MAX) : given;
  float base = fmaxf(m, sink);
  base = base == -INFINITY ? 0.f : base;
  if (sinks) l = l * exp2_fast(m - base) + exp2_fast(sink - base);
  e.mul = l == 0.f ? 0.f : __fdividef(exp2_fast(m - base), l);  // (nothing has any weight: zeros, as without a token)
  e.lse = fmaf(__log2f(l), 0.693147181f, sink > m ? given : base * 0.693147181f);
  return e;
}

// 8 dims of a row's joined states.  add() takes states first, first + step, .. below
// end, N at a time: their loads do not wait for one another, so that a join
// takes one trip to memory per N states (maxima first and sums then took 5 us for
// two states of 16 x 256; FAR: written by another block, read past L1).
struct Joined {
  float m = -INFINITY, l = 0.f, y[8] = {};
  bool gone = false;  // a block that gave up is among them

  template <int N, bool FAR, class At>
  __device__ __forceinline__ void add(int first, int end, int step, At at, int row, int rows, int sums) {
    auto ld = [](const float *p) { return FAR ? __ldcg(p) : *p; };
    auto ld4 = [](const float *p) {
      return FAR ? __ldcg(reinterpret_cast<const float4 *>(p)) : *reinterpret_cast<const float4 *>(p);
    };
#pragma unroll 1
    for (int i = first; i < end; i += N * step) {
      float ms[N], ls[N];
      float4 z[N][2];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        ms[k] = -INFINITY;
        ls[k] = 0.f;
        z[k][0] = z[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i + k * step < end) {
          const float *st = at(i + k * step);
          ms[k] = ld(st + row);
          ls[k] = ld(st + rows + row);
          z[k][0] = ld4(st + sums);
          z[k][1] = ld4(st + sums + 4);
        }
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        top = fmaxf(top, ms[k]);
        gone |= ls[k] < 0.f;
      }
      const float base = top == -INFINITY ? 0.f : top, fade = exp2_fast(m - base);
      m = top;
      l *= fade;
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= fade;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float w = exp2_fast(ms[k] - base);
        l = fmaf(w, ls[k], l);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          y[4 * h] = fmaf(w, z[k][h].x, y[4 * h]);
          y[4 * h + 1] = fmaf(w, z[k][h].y, y[4 * h + 1]);
          y[4 * h + 2] = fmaf(w, z[k][h].z, y[4 * h + 2]);
          y[4 * h + 3] = fmaf(w, z[k][h].w, y[4 * h + 3]);
        }
      }
    }
  }
};
__device__ __forceinline__ void store8(uint8_t *out, const float (&y)[8], float mul) {
  *reinterpret_cast<uint4 *>(out) =
      make_uint4(pack_bf16x2(y[0] * mul, y[1] * mul), pack_bf16x2(y[2] * mul, y[3] * mul),
                 pack_bf16x2(y[4] * mul, y[5] * mul), pack_bf16x2(y[6] * mul, y[7] * mul));
}

// ------------------------------------------------------------------ kernel

// What a stage of a ring holds (written for the first step of a unit or of a warp's range).
struct Step {
  int seq, unit, pos, len;  // sequence, unit, first token of the step, tokens of the sequence
};
// At its range's end a warp's state takes the place of its ring, two stages at least.
constexpr bool state_fits(int type, int dim, bool any, int tt, int rows) {
  for (int d = any ? 16 : dim; d <= dim; d += 16)
    if (state_floats(rows, d) * 4 > 2 * tt * kv_tile_bytes(type, d)) return false;
  return true;
}

// What the warps of a block share beside their rings.
struct AttendShared {
  uint64_t full[kAttMaxWarps][kAttMaxStages];
  Step held[kAttMaxWarps][kAttMaxStages];
  // a warp's first slot, from its sequence's first, and that sequence and its length; last entry: the block's last slot
  longlong2 scan[kAttMaxWarps];
  long long from[kAttMaxWarps + 1];
  int2 start[kAttMaxWarps + 1];
  int4 piece[2 * kAttMaxWarps];  // [2 warp + which]: {sequence (-1: none), unit, cut before 1 / after 2, -}
  const float *where[2 * kAttMaxWarps];
  int order[2 * kAttMaxWarps], run[2 * kAttMaxWarps + 1];  // pieces in order; where each unit's run starts
  int n_runs, dead_block;
  int2 to_join[2];  // {first block, blocks} of units that this block was the last to work on
};
constexpr int kAttStatic = 3584;  // kept free of rings for it
static_assert(sizeof(AttendShared) <= kAttStatic, "the shared memory beside the rings");

// A unit as its key head and the first of its query heads in that head's group, in one number.
__device__ __forceinline__ int pack_unit(int kvh, int h0) { return kvh << 16 | h0; }
__device__ __forceinline__ int unit_kvh(int unit) { return unit >> 16; }
__device__ __forceinline__ int unit_h0(int unit) { return unit & 0xffff; }

// a / b, without the long division where 32 bits do (a call: it is used in places that run once).
static __device__ __noinline__ unsigned long long quotient(unsigned long long a, unsigned long long b) {
  return (a | b) >> 32 ? a / b : (unsigned)a / (unsigned)b;
}

// DIM: the head's width, or with ANY the largest of a range of multiples of 16 (kv.dim is the width).
// TT: tiles of 16 tokens per step.  WARPS: most warps of a block.  NT: 8 NT query heads to a unit.
template <int TYPE, int DIM, bool ANY, int TT, int WARPS, int NT>
__global__ void __launch_bounds__(WARPS * 32, 1) attend_kernel(KvView kv, KvSeqs s, AttendArgs a) {
  constexpr int ES = kv_elt(TYPE);
  constexpr int ROWS = 8 * NT;          // query heads of a unit
  constexpr int NB = DIM / 16;          // blocks of 16 dims
  const int dim = ANY ? kv.dim : DIM, nb = ANY ? kv.dim / 16 : NB;
  const int row_bytes = dim * ES, chunks = row_bytes / 16;
  constexpr int kStep = kTileTokens * TT;  // tokens of a step
  const int tile_bytes = kv_tile_bytes(TYPE, dim), stage_bytes = TT * tile_bytes;

  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ AttendShared sh;
  auto &full = sh.full;
  auto &held = sh.held;
  auto &scan = sh.scan;
  auto &from = sh.from;
  auto &start = sh.start;
  auto &piece = sh.piece;
  auto &where = sh.where;
  auto &order = sh.order;
  auto &run = sh.run;
  int &n_runs = sh.n_runs, &dead_block = sh.dead_block;
  auto &to_join = sh.to_join;
  static_assert(state_fits(TYPE, DIM, ANY, TT, ROWS), "a state has to fit into the smallest ring");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_warps = blockDim.x >> 5;
  const int floats = state_floats(a.rows, dim);

  if (lane < a.n_stages) mbar_init(&full[warp][lane], 1);
  fence_mbar_init();
  if (tid < 2 * kAttMaxWarps) piece[tid] = make_int4(-1, 0, 0, 0);
  if (tid == 0) dead_block = 0;
  griddep_wait();
  griddep_launch_dependents();

  // ---- this block's and this warp's range of the flat list
  const int per = (s.n + blockDim.x - 1) / blockDim.x;
  const int s0 = min(s.n, tid * per), s1 = min(s.n, s0 + per);
  // (slots of a unit, summed, and sequences with a token, counted in the bits above)
  constexpr int kCountAt = 42;
  long long mine = 0;
  unsigned longest = 0;
  int last_len = 0;
#pragma unroll 1
  for (int i = s0; i < s1; ++i) {
    last_len = seq_len(kv, s, i);
    const unsigned n = unit_slots(last_len, a.window, TT);
    mine += n | (n ? 1ll << kCountAt : 0);
    longest = max(longest, n);
  }
  long long before = mine;  // inclusive scan over the block
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(~0u, before, d);
    if (lane >= d) before += x;
  }
  longest = __reduce_max_sync(~0u, longest);
  if (lane == 31) scan[warp] = make_longlong2(before, longest);
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int i = 0; i < kAttMaxWarps; ++i)
    if (i < n_warps) {
      const longlong2 x = scan[i];
      if (i < warp) before += x.x;
      total += x.x;
      longest = max(longest, (unsigned)x.y);
    }
  constexpr long long kSlotBits = (1ll << kCountAt) - 1;
  long long *prefix = reinterpret_cast<long long *>(smem);  // [threads], before the rings are in use
  int *only = reinterpret_cast<int *>(prefix + blockDim.x);  // lengths, where a thread has one sequence
  prefix[tid] = before - mine;
  only[tid] = last_len;
  __syncthreads();

  // The sequence at place y of the list of slots (or of sequences with a token),
  // by a whole warp: the last thread whose share starts at or before y, then its
  // sequences.  before: the slots in front of it.
  auto find = [&](long long y, bool by_count, int &seq, int &len, long long &before) {
    auto key = [&](long long x) { return by_count ? x >> kCountAt : x & kSlotBits; };
    int t = __popc(__ballot_sync(~0u, key(prefix[lane * n_warps]) <= y)) - 1;
    t = t * n_warps + __popc(__ballot_sync(~0u, lane < n_warps && key(prefix[min(t * n_warps + lane, (int)blockDim.x - 1)]) <= y)) - 1;
    long long sum = prefix[t];
    if (per == 1) {  // (the usual case: at most as many sequences as threads)
      seq = t;
      len = only[t];
      before = sum & kSlotBits;
      return;
    }
    const int end = min(s.n, (t + 1) * per);
#pragma unroll 1
    for (int i0 = t * per; i0 < end; i0 += 32) {
      const int l = i0 + lane < end ? seq_len(kv, s, i0 + lane) : 0;
      const unsigned n = unit_slots(l, a.window, TT);
      const long long own = n | (n ? 1ll << kCountAt : 0);
      long long upto = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(~0u, upto, d);
        if (lane >= d) upto += x;
      }
      const unsigned past = __ballot_sync(~0u, key(sum + upto) > y);
      if (past) {
        const int at = __ffs(past) - 1;
        seq = i0 + at;
        len = __shfl_sync(~0u, l, at);
        before = __shfl_sync(~0u, (sum + upto - own) & kSlotBits, at);
        return;
      }
      sum += __shfl_sync(~0u, upto, 31);
    }
  };

  const unsigned long long slots_all = (unsigned long long)(total & kSlotBits) * a.units;
  const bool too_long = slots_all > (unsigned long long)gridDim.x << kMaxSlotsLog2;
  const unsigned long long units_all = (unsigned long long)(total >> kCountAt) * a.units;
  // A unit cut between blocks costs their last one kCutSteps steps' time or so, in each
  // warp.  While blocks of whole units are longer by less than that, none is cut
  // (attention alone, whole and cut: 16 requests of up to 100 tokens 9.2 and 12.4
  // us, 256 requests with a window of 128 20.3 and 21.4; 64 requests of 200 to 4000
  // tokens 317 and 181, 37 of 5 to 9001 with 16 heads of 256 143 and 50, which are cut).
  const unsigned long long most_units = quotient(units_all + gridDim.x - 1, gridDim.x);  // of a block
  const bool by_units = most_units * longest * gridDim.x <= slots_all + (unsigned long long)kCutSteps * n_warps * gridDim.x;
  // (two slots at least to a block, so that it has a step: the join counts on
  // every block in a row having a part)
  const unsigned long long items = by_units ? units_all : slots_all;
  const unsigned blocks = (unsigned)min((unsigned long long)gridDim.x, by_units ? items : items / 2);
  const unsigned long long each = quotient(items, max(blocks, 1u));  // items of a block; the first `more` have one more
  const unsigned more = (unsigned)(items - each * blocks);
  long long b0 = each * blockIdx.x + min(blockIdx.x, more);
  int slots = blockIdx.x < blocks && !too_long ? (int)each + (blockIdx.x < more) : 0;
  if (too_long && tid == 0) set_status(kv.status, LORA_ERR_BAD_ID);
  if (by_units) {  // from units to slots: warp 0 the first unit's start, warp 1 the last one's end
    if (slots > 0 && warp < 2) {
      const long long u = warp ? b0 + slots - 1 : b0, y = quotient(u, a.units);
      int seq = 0, len = 0;
      long long p = 0;
      find(y, true, seq, len, p);
      if (lane == 0) from[warp] = p * a.units + (u - y * a.units + warp) * unit_slots(len, a.window, TT);
    }
    __syncthreads();
    b0 = from[0];
    slots = slots ? (int)(from[1] - b0) : 0;
    __syncthreads();
  }
  const int wq = slots / n_warps, wr = slots - wq * n_warps;
#pragma unroll 1
  for (int w = warp; w <= n_warps; w += n_warps) {  // this warp's first slot; warp 0: the block's last one too
    const int at = w < n_warps ? wq * w + min(w, wr) : slots - 1;
    if (at >= slots || at < 0) continue;
    const long long x = b0 + at, y = quotient(x, a.units);
    int seq = 0, len = 0;
    long long p = 0;
    find(y, false, seq, len, p);
    if (lane == 0) {
      start[w] = make_int2(seq, len);
      from[w] = x - p * a.units;
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (prefix, before the copies into the rings)
  __syncthreads();
  const int count = wq + (warp < wr);  // this warp's slots

  uint8_t *ring = smem + (size_t)warp * a.n_stages * stage_bytes;
  if (count > 0) {
    // ---- fetching side: the next step to fetch, and pages of up to 32 tiles
    int left = count;  // slots not yet passed
    int fetched = 0;   // steps fetched or being so
    int fseq = start[warp].x, flen = start[warp].y;
    int fkvh, fh0, fpos;  // the unit's key head and first query head; first token of the step
    bool fnew = true;     // the step to fetch is the first of a unit or of the range
    bool own_slot;        // the unit's own slot is to be passed first
    {
      const int n = unit_slots(flen, a.window, TT), unit = (int)quotient(from[warp], n);
      const int slot = (int)(from[warp] - (long long)unit * n);
      own_slot = slot == 0;
      fpos = (first_token(flen, a.window) / kStep + max(slot - 1, 0)) * kStep;
      fkvh = a.head_groups == 1 ? unit : unit / a.head_groups;
      fh0 = (unit - fkvh * a.head_groups) * ROWS;
    }
    const bool starts_inside = fpos > first_token(flen, a.window);  // of its unit
    unsigned bad_tiles = 0;     // bits stage * TT ..: tiles of a stage that are on no page of the cache
    const long long head_stride = kv_head_stride(kv);
    const uint8_t *fhead = kv.base + fkvh * head_stride;
    // a step's tiles lie in one page, one behind the other, unless pages are shorter
    const bool one_copy = TT == 1 || (1 << kv.log2_page) >= kStep;
    // lane i: page of the sequence's tile base + i, or -1
    auto load_pages = [&](int seq, int len, int base) {
      const int tok = (base + lane) * kTileTokens;
      return tok < len ? __ldg(s.table + (long long)seq * s.max_pages + (tok >> kv.log2_page)) : -1;
    };
    int pbase = fpos / kTileTokens & ~31, pages = load_pages(fseq, flen, pbase);
    // the sequence after: its length is read when this one begins, its first pages when this one's last unit does
    int nlen = fseq + 1 < s.n ? __ldg(s.lens + fseq + 1) : 0, npages = 0;
    auto load_next = [&]() {
      if (fkvh != kv.heads - 1 || fh0 + ROWS < a.group || fseq + 1 >= s.n) return;
      nlen = valid_len(kv, s, nlen);
      npages = load_pages(fseq + 1, nlen, first_token(nlen, a.window) / kStep * TT & ~31);
    };
    load_next();

    auto fetch = [&](int stage) {
      if (own_slot) {
        --left;
        own_slot = false;
      }
      if (left <= 0) return;
      --left;
      ++fetched;
      const int t = fpos / kTileTokens;
      if ((t & ~31) != pbase) {
        pbase = t & ~31;
        pages = load_pages(fseq, flen, pbase);
      }
      // tiles [t0, t1) of the step, by lane 0 in one copy or by a lane each
      const int t0 = max(first_token(flen, a.window) / kTileTokens - t, 0);
      const int t1 = min((flen - fpos + kTileTokens - 1) / kTileTokens, TT);
      const int tile = one_copy ? t0 : t0 + lane;
      const int page = __shfl_sync(~0u, pages, (t + tile) & 31);
      const long long at = kv_tile_offset(kv, page, fpos + tile * kTileTokens);
      bool copy = at >= 0 && lane < (one_copy ? 1 : t1 - t0);
      int n = at >= 0 ? t1 - t0 : 0;
      if (TT > 1 && !one_copy) n = __popc(__ballot_sync(~0u, copy));
      if (lane == 0) {
        if (fnew) held[warp][stage] = {fseq, pack_unit(fkvh, fh0), fpos, flen};
        if (a.stall != kStallAll) mbar_arrive_expect_tx(&full[warp][stage], n * tile_bytes);
      }
      if (n < t1 - t0) {
        const unsigned ok = TT > 1 && !one_copy ? __ballot_sync(~0u, copy) << t0 : 0u;
        bad_tiles |= (((1u << t1) - (1u << t0)) & ~ok) << (stage * TT);
        if (lane == 0) set_status(kv.status, LORA_ERR_BAD_ID);
      }
      __syncwarp();
      if (copy && a.stall != kStallAll)
        bulk_g2s(ring + stage * stage_bytes + tile * tile_bytes, fhead + at, one_copy ? n * tile_bytes : tile_bytes,
                 &full[warp][stage]);
      fpos += kStep;
      fnew = fpos >= flen;
      if (fnew) {
        own_slot = true;
        fh0 += ROWS;
        if (fh0 >= a.group) {
          fh0 = 0;
          ++fkvh;
          fhead += head_stride;
        }
        if (fkvh == kv.heads) {
          fkvh = 0;
          fhead = kv.base;
          if (left > 1) {  // (another step is to come)
            ++fseq;
            flen = valid_len(kv, s, nlen);
            pages = npages;
            pbase = first_token(flen, a.window) / kStep * TT & ~31;
#pragma unroll 1
            while (flen == 0) {
              ++fseq;
              flen = seq_len(kv, s, fseq);
              pbase = -1;
            }
            nlen = fseq + 1 < s.n ? __ldg(s.lens + fseq + 1) : 0;
          }
        }
        fpos = first_token(flen, a.window) / kStep * kStep;
        load_next();
      }
    };

    // ---- computing side
    const uint32_t ring32 = smem_u32(ring);
    const int g = lane >> 2, j2 = 2 * (lane & 3);  // of a product: its row (token, dim) and its pair of columns (heads)
    const int r8 = lane & 7, mat = lane >> 3;      // this lane's row and matrix of an ldmatrix
    const int low = chunks & -chunks, grp = low < 8 ? low : 8;
    const int sw = (r8 / (8 / grp)) & (grp - 1);  // its rows' chunk permutation (rows r8 and r8 + 8 share it)
    // K: (tokens 0-7 | 8-15) x (chunk | next chunk); V, transposed: the same for 8 bits, for bf16 chunks first
    const uint32_t k_row = ((mat & 1) * 8 + r8) * row_bytes;
    const uint32_t v_row = (kTileTokens + (TYPE == LORA_KV_BF16 ? mat >> 1 : mat & 1) * 8 + r8) * row_bytes;
    const int k_c = mat >> 1, v_c = TYPE == LORA_KV_BF16 ? mat & 1 : mat >> 1;

    uint32_t qa[NT][2 * NB];
    float qs[NT][2];  // what a score is multiplied by: the softmax's scale and q's
    unsigned fine = 0;  // (8 bits) not 0: the unit's scores are formed in bf16; byte h: exponent of what row 8 h + g of q is divided by
    float o[NT][NB][4], m[NT][2], l[NT][2];
    float w[NT][2];  // (8 bits) reference of the weights times V's scales, from m
    int cseq = -1, cunit = -1, cpos = 0, clen = 0, cfirst = 0;  // of the step to compute; cfirst: the unit's first token
    bool cut_before = false, cnew = true;
    int stage = 0, fstage = 0;
    uint32_t phase = 0;

    // q as the products' B operand: columns = heads, rows = dims in the order of the K operand
    auto load_q = [&]() {
      const int kvh = unit_kvh(cunit), h0 = unit_h0(cunit), j = lane & 3;
      bool more = false;
      unsigned exps = 0;
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        const bool live = h0 + g + 8 * h < a.group;
        const uint8_t *q = a.q + cseq * a.ldq + (long long)(kvh * a.group + h0 + g + 8 * h) * dim * 2;
        uint32_t(&u)[2 * NB] = qa[h];  // bf16: dims 16 b + 2 j, + 1, + 8, + 9; 8 bits: dims 16 b + 4 j ..
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          u[2 * b] = u[2 * b + 1] = 0;
          if (!live || (ANY && b >= nb)) continue;
          if (TYPE == LORA_KV_BF16) {
            u[2 * b] = __ldg(reinterpret_cast<const uint32_t *>(q + b * 32 + j * 4));
            u[2 * b + 1] = __ldg(reinterpret_cast<const uint32_t *>(q + b * 32 + j * 4 + 16));
          } else {
            const uint2 x = __ldg(reinterpret_cast<const uint2 *>(q + b * 32 + j * 8));
            u[2 * b] = x.x;
            u[2 * b + 1] = x.y;
          }
        }
        if (TYPE == LORA_KV_BF16) {
          qs[h][0] = qs[h][1] = a.scale2;
          continue;
        }
        uint32_t top = 0, low = ~0u;  // bits of the head's largest |q|, and of the least but 0 (less 1), two by two
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) {
          top = __vmaxu2(top, u[i] & 0x7fff7fffu);
          low = __vminu2(low, ((u[i] | 0x80008000u) - 0x00010001u) ^ 0x80008000u);
        }
        top = max(top & 0xffffu, top >> 16);
        low = min(low & 0xffffu, low >> 16);
        top = max(top, __shfl_xor_sync(~0u, top, 1));
        top = max(top, __shfl_xor_sync(~0u, top, 2));
        more |= (int)low < (int)(top & 0x7f80u) - (kFine << 7);
        const float amax = fmaxf(__uint_as_float(top << 16), 0x1p-111f);  // (a NaN is lost here and comes back below)
        const float two = __uint_as_float(__float_as_uint(amax) & 0x7f800000u);  // 2^E, 2^E <= amax
        const float mul = __uint_as_float(__float_as_uint(kQTop) + __float_as_uint(1.f) - __float_as_uint(two));  // kQTop / two
        exps |= __float_as_uint(two) >> 23 << (8 * h);
        const float mine = top >= 0x7f80u ? __int_as_float(0x7fc00000) : two * (a.scale2 / kQTop);
        qs[h][0] = __shfl_sync(~0u, mine, 4 * j2);
        qs[h][1] = __shfl_sync(~0u, mine, 4 * j2 + 4);
#pragma unroll
        for (int b = 0; b < NB; ++b) {  // as key_codes_to_f16 pairs the dims
          const float x0 = bf16_lo(u[2 * b]) * mul, x1 = bf16_hi(u[2 * b]) * mul;
          const float x2 = bf16_lo(u[2 * b + 1]) * mul, x3 = bf16_hi(u[2 * b + 1]) * mul;
          u[2 * b] = TYPE == LORA_KV_E4M3 ? pack_f16x2(x0, x1) : pack_f16x2(x0, x2);
          u[2 * b + 1] = TYPE == LORA_KV_E4M3 ? pack_f16x2(x2, x3) : pack_f16x2(x1, x3);
        }
      }
      fine = __any_sync(~0u, more) ? exps : 0;
      if (fine) {
#pragma unroll
        for (int h = 0; h < NT; ++h) qs[h][0] *= kQTop, qs[h][1] *= kQTop;
      }
    };

    // (the first iterations fill the ring: one place in the code for each part)
#pragma unroll 1
    for (int i = 1 - a.n_stages;; ++i) {
      asm volatile("" : "+r"(i));  // (one copy of the loop's body, not one for the filling)
      fetch(fstage);
      if (++fstage == a.n_stages) fstage = 0;
      if (i < 0) continue;
      int leaving = i == fetched ? 2 : cnew;  // (opaque, for the same reason)
      asm volatile("" : "+r"(leaving));
      if (leaving) {
        if (cseq >= 0) {
          // The unit's state leaves the registers: as its result when the warp
          // has seen all of it, else as a piece to be joined (at the range's end
          // the ring is free for it).
          const bool cut_after = leaving == 2 && !cnew;
          const bool whole = !cut_before && !cut_after;
          const int kvh = unit_kvh(cunit), h0 = unit_h0(cunit);
          float *state = leaving == 2 ? reinterpret_cast<float *>(ring) : a.first_in_smem
                             ? reinterpret_cast<float *>(smem + a.first_in_smem) + warp * floats
                             : a.first + ((size_t)blockIdx.x * kAttMaxWarps + warp) * floats;
          if (!whole && lane == 0) {
            const int k = 2 * warp + (cut_before ? 0 : 1);
            piece[k] = make_int4(cseq, cunit, (cut_before ? 1 : 0) | (cut_after ? 2 : 0), 0);
            where[k] = state;
          }
#pragma unroll
          for (int h = 0; h < NT; ++h) {
            float mul[2], half[2];  // (8 bits: 2^w, which may pass the exponent's range, in two halves)
            bool on[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              l[h][e] += __shfl_xor_sync(~0u, l[h][e], 4);
              l[h][e] += __shfl_xor_sync(~0u, l[h][e], 8);
              l[h][e] += __shfl_xor_sync(~0u, l[h][e], 16);
              const int r = 8 * h + j2 + e, hd = kvh * a.group + h0 + r;
              on[e] = r < a.rows && h0 + r < a.group;
              half[e] = TYPE == LORA_KV_BF16 ? 1.f : exp2_fast(0.5f * w[h][e]);
              mul[e] = half[e];
              if (!on[e]) continue;
              if (whole) {
                const Ends x = finish(a.sinks, hd, m[h][e], l[h][e]);
                mul[e] *= x.mul;
                if (a.lse && g == 0) a.lse[(long long)cseq * a.n_heads + hd] = x.lse;
              } else if (g == 0) {
                state[r] = m[h][e];
                state[a.rows + r] = l[h][e];
              }
            }
            const int r = 8 * h + j2;
            float *sums = state + state_head(a.rows) + r * dim;
            uint8_t *out = a.out + cseq * a.ldo + (long long)(kvh * a.group + h0 + r) * dim * 2;
            // a thread's two neighbouring dims of each of its two heads; 8 bits:
            // rows g and g + 8 are dims 2 g and 2 g + 1; bf16: dims g and g + 8, and
            // neighbouring rows trade one
            const int d0 = TYPE != LORA_KV_BF16 ? 2 * g : g & 1 ? 7 + g : g;
            auto pair_of = [&](int b, int e) {
              float2 x = make_float2(o[h][b][e], o[h][b][2 + e]);
              if (TYPE == LORA_KV_BF16) {
                const float got = __shfl_xor_sync(~0u, g & 1 ? x.x : x.y, 4);
                x = g & 1 ? make_float2(got, x.y) : make_float2(x.x, got);
              }
              if (TYPE != LORA_KV_BF16) x = make_float2(x.x * half[e], x.y * half[e]);
              return make_float2(x.x * mul[e], x.y * mul[e]);
            };
            if (whole) {
#pragma unroll
              for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  if (ANY && b >= nb) continue;
                  const float2 x = pair_of(b, e);
                  if (on[e]) *reinterpret_cast<uint32_t *>(out + (e * dim + 16 * b + d0) * 2) = pack_bf16x2(x.x, x.y);
                }
            } else {
#pragma unroll
              for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  if (ANY && b >= nb) continue;
                  const float2 x = pair_of(b, e);
                  if (on[e]) *reinterpret_cast<float2 *>(sums + e * dim + 16 * b + d0) = x;
                }
            }
          }
        }
        if (leaving == 2) break;
        cut_before = i == 0 && starts_inside;
        const Step st = held[warp][stage];
        cseq = st.seq;
        cunit = st.unit;
        cpos = st.pos;
        clen = st.len;
        cfirst = first_token(clen, a.window);
#pragma unroll
        for (int h = 0; h < NT; ++h) {
          m[h][0] = m[h][1] = -INFINITY;
          w[h][0] = w[h][1] = -INFINITY;
          l[h][0] = l[h][1] = 0.f;
#pragma unroll
          for (int b = 0; b < NB; ++b) o[h][b][0] = o[h][b][1] = o[h][b][2] = o[h][b][3] = 0.f;
        }
        load_q();
        {  // the next unit's q, towards this SM: the rows behind, or the next sequence's first
          const int kvh = unit_kvh(cunit), h0 = unit_h0(cunit);
          const bool more_heads = h0 + ROWS < a.group, last = kvh == kv.heads - 1 && !more_heads;
          const uint8_t *q = last ? a.q + (cseq + 1) * a.ldq
                                  : a.q + cseq * a.ldq + (long long)(kvh * a.group + min(h0 + ROWS, a.group)) * dim * 2;
          const int bytes = (more_heads ? min(a.rows, a.group - h0 - ROWS) : a.rows) * dim * 2;
          if (!last || cseq + 1 < s.n)
#pragma unroll 1
            for (int x = lane * 128; x < bytes; x += 32 * 128) asm volatile("prefetch.global.L1 [%0];" ::"l"(q + x));
        }
      }
      // One verdict a warp: its lanes read their clocks one by one, and where a copy
      // lands as the limit passes, some see it and others do not.
      bool landed = mbar_wait_bounded(&full[warp][stage], phase, kv.status, a.wait_ns);
      if (a.stall == kStallLane + lane && i >= 2) landed = false;
      if (!__all_sync(~0u, landed)) {
        // Copies in flight (steps fetched and not computed) must land before the block
        // ends: they get the limit once more, all together.
        const long long t0 = clock64();
        const int flying = a.stall == kStallAll ? 0 : fetched - i;
#pragma unroll 1
        for (int k = 0; k < flying; ++k) {
          const long long spent = (clock64() - t0) / 2;  // (ns at 2 GHz, as the wait counts them)
          (void)mbar_wait_bounded(&full[warp][stage], phase, kv.status, max((long long)a.wait_ns - spent, 0ll));
          if (++stage == a.n_stages) {
            stage = 0;
            phase ^= 1;
          }
        }
        __syncwarp();
        if (lane == 0) {
          dead_block = 1;
          set_status(kv.status, LORA_ERR_TIMEOUT);
        }
        break;
      }
      const uint32_t st32 = ring32 + stage * stage_bytes;
      uint8_t *stp = ring + stage * stage_bytes;
      // tokens of the step that count: [lo, hi) of its 16 TT, without those on bad pages
      const int lo = cfirst - cpos, hi = clen - cpos;
      const unsigned bad = bad_tiles >> (stage * TT) & ((1u << TT) - 1u);
      const bool partial = lo > 0 || hi < kStep || bad;
      bad_tiles &= ~(((1u << TT) - 1u) << (stage * TT));
      cpos += kStep;
      cnew = cpos >= clen;
      if (TYPE != LORA_KV_INT8 && partial) {
        // weight 0 times what lies there must be 0: clear V's rows outside (int8 has no NaN)
#pragma unroll 1
        for (int x = lane; x < kStep * chunks; x += 32) {
          const int t = x / chunks;
          if (t >= lo && t < hi && !(bad >> (t / kTileTokens) & 1)) continue;
          *reinterpret_cast<uint4 *>(stp + (t / kTileTokens) * tile_bytes + (kTileTokens + t % kTileTokens) * row_bytes +
                                     (x - t * chunks) * 16) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }

      // ---- scores: [16 TT tokens] x [heads]; rows g and g + 8 of each tile, columns j2 and j2 + 1
      float c[TT][NT][4];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint32_t k32 = st32 + t * tile_bytes + k_row;
        float d[NT][4] = {};  // a second sum for the odd blocks: a shorter chain
#pragma unroll
        for (int h = 0; h < NT; ++h) c[t][h][0] = c[t][h][1] = c[t][h][2] = c[t][h][3] = 0.f;
        if (TYPE == LORA_KV_BF16) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            if (ANY && b >= nb) continue;
            uint32_t k[4];
            ldsm4(k, k32 + (((2 * b + k_c) ^ sw) << 4));
#pragma unroll
            for (int h = 0; h < NT; ++h)
              mma16816(b & 1 ? d[h] : c[t][h], k[0], k[1], k[2], k[3], qa[h][2 * b], qa[h][2 * b + 1]);
          }
        } else {
          if (!fine) {
#pragma unroll
            for (int p = 0; p < (NB + 1) / 2; ++p) {
              if (ANY && 2 * p >= nb) continue;
              uint32_t w[4];  // (tokens 0-7 | 8-15) x (block 2p | 2p + 1)
              ldsm4(w, k32 + (((2 * p + k_c) ^ sw) << 4));
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int b = 2 * p + x;
                if (b >= NB || (ANY && b >= nb)) continue;
                uint32_t k0, k1, k2, k3;
                key_codes_to_f16<TYPE>(w[2 * x], k0, k2);
                key_codes_to_f16<TYPE>(w[2 * x + 1], k1, k3);
#pragma unroll
                for (int h = 0; h < NT; ++h) mma_f16(x ? d[h] : c[t][h], k0, k1, k2, k3, qa[h][2 * b], qa[h][2 * b + 1]);
              }
            }
          } else {  // (rare: q is read again, and nothing of it kept in registers)
            const uint8_t *q = a.q + cseq * a.ldq + ((long long)(unit_kvh(cunit) * a.group + unit_h0(cunit)) * dim + 4 * (lane & 3)) * 2;
#pragma unroll 1
            for (int b = 0; b < nb; ++b) {
              uint32_t w[4], k0, k1, k2, k3;
              ldsm4(w, k32 + ((((b & ~1) + k_c) ^ sw) << 4));
              key_codes_to_bf16<TYPE>(b & 1 ? w[2] : w[0], k0, k2);
              key_codes_to_bf16<TYPE>(b & 1 ? w[3] : w[1], k1, k3);
#pragma unroll
              for (int h = 0; h < NT; ++h) {
                const float one = 1.f / __uint_as_float((fine >> (8 * h) & 255u) << 23), up = TYPE == LORA_KV_E4M3 ? kFineScale : 1.f;
                uint2 u = make_uint2(0, 0);
                if (unit_h0(cunit) + g + 8 * h < a.group)
                  u = __ldg(reinterpret_cast<const uint2 *>(q + ((g + 8 * h) * dim + b * 16) * 2));
                const float x0 = bf16_lo(u.x) * one * up, x1 = bf16_hi(u.x) * one * up;
                const float x2 = bf16_lo(u.y) * one * up, x3 = bf16_hi(u.y) * one * up;
                mma16816(d[h], k0, k1, k2, k3, TYPE == LORA_KV_E4M3 ? pack_bf16x2(x0, x1) : pack_bf16x2(x0, x2),
                         TYPE == LORA_KV_E4M3 ? pack_bf16x2(x2, x3) : pack_bf16x2(x1, x3));
              }
            }
          }
        }
        float ks[2] = {1.f, 1.f};
        if (TYPE != LORA_KV_BF16) {
          const uint8_t *sc = stp + t * tile_bytes + 2 * kTileTokens * row_bytes;
          ks[0] = *reinterpret_cast<const float *>(sc + g * 4);
          ks[1] = *reinterpret_cast<const float *>(sc + g * 4 + 32);
        }
#pragma unroll
        for (int h = 0; h < NT; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            c[t][h][e] += d[h][e];
            c[t][h][e] *= TYPE == LORA_KV_BF16 ? qs[h][e & 1] : ks[e >> 1] * qs[h][e & 1];
          }
      }

      // ---- weights
      float lv[TT][2];  // log2 of V's scales
      if (TYPE != LORA_KV_BF16) {
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const uint8_t *sc = stp + t * tile_bytes + 2 * kTileTokens * row_bytes + kTileTokens * 4;
          lv[t][0] = log2_fast(*reinterpret_cast<const float *>(sc + g * 4));
          lv[t][1] = log2_fast(*reinterpret_cast<const float *>(sc + g * 4 + 32));
        }
      }
      if (partial) {
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = t * kTileTokens + g + 8 * e;
            if (j < lo || j >= hi || (bad >> t & 1)) {
#pragma unroll
              for (int h = 0; h < NT; ++h) c[t][h][2 * e] = c[t][h][2 * e + 1] = -INFINITY;
              if (TYPE != LORA_KV_BF16) lv[t][e] = -INFINITY;
            }
          }
      }
      // m is a reference, up to kSlack above the running maximum: while no score
      // passes it, nothing is exchanged and nothing rescaled, and no weight is above 1
      // (V may be as large as its type allows).  The
      // values' sums have one of their own: with 8 bits m + w, by the weights times V's
      // scales (in logarithms: their product may pass the exponent's range), which
      // leaves the largest of those between 2^kWeight and 2^(kWeight + kSlack).
      // (By V's largest scale alone a token with a far larger V and next to no
      // weight would take the others' bits.)  Logarithms are added to scores less m:
      // a large score itself has no bits left for them.
      float mx[NT][2];
      bool moved = false;
      auto finite = [](float x) { return x == -INFINITY ? 0.f : x; };
      auto weighted_max = [&](int h, int e, float base) {
        float x = -INFINITY;
#pragma unroll
        for (int t = 0; t < TT; ++t) x = fmaxf(x, fmaxf(c[t][h][e] - base + lv[t][0], c[t][h][e + 2] - base + lv[t][1]));
        return x;
      };
#pragma unroll
      for (int h = 0; h < NT; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[h][e] = c[0][h][e];
#pragma unroll
          for (int t = 0; t < TT; ++t) mx[h][e] = fmaxf(mx[h][e], fmaxf(c[t][h][e], c[t][h][e + 2]));
          moved |= mx[h][e] > m[h][e];
          if (TYPE != LORA_KV_BF16) moved |= weighted_max(h, e, finite(m[h][e])) > w[h][e] + (kWeight + kSlack);
        }
      if (__any_sync(~0u, moved)) {
#pragma unroll
        for (int h = 0; h < NT; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            auto highest = [&](float x) {
              x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
              x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
              return fmaxf(x, __shfl_xor_sync(~0u, x, 16));
            };
            const float top = fmaxf(highest(mx[h][e]) + kSlack, m[h][e]), by = m[h][e] - finite(top);
            m[h][e] = top;
            float alpha = exp2_fast(by);
            l[h][e] *= alpha;
            if (TYPE != LORA_KV_BF16) {
              const float was = w[h][e] + by;
              w[h][e] = fmaxf(highest(weighted_max(h, e, finite(top))) - kWeight, was);
              alpha = exp2_fast(was - finite(w[h][e]));
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              if (ANY && b >= nb) continue;
              o[h][b][e] *= alpha;
              o[h][b][e + 2] *= alpha;
            }
          }
      }
      // bf16: the weights as two terms, hi with the type's leading bits (cut, so
      // that the rest is exact) and the rest's leading bits: one term would add an
      // error of the size of the result's own rounding.  8 bits: the weights times
      // V's scales as fp16, whose 11 bits leave a fraction of that; the largest is
      // 2^kWeight or more, so that one is off by at most 2^-11 of itself or 2^-36 of
      // the largest.  Each turned: a thread then has two tokens of head g.
      constexpr int TERMS = TYPE == LORA_KV_BF16 ? 2 : 1;
      uint32_t pw[TERMS][TT][NT][2];
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        const float base[2] = {finite(m[h][0]), finite(m[h][1])}, wbase[2] = {finite(w[h][0]), finite(w[h][1])};
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // tokens g and g + 8
            const float x0 = c[t][h][2 * e] - base[0], x1 = c[t][h][2 * e + 1] - base[1];
            const float p0 = exp2_fast(x0), p1 = exp2_fast(x1);
            l[h][0] += p0;
            l[h][1] += p1;
            if (TYPE == LORA_KV_BF16) {
              const uint32_t hi2 = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
              pw[0][t][h][e] = turn(hi2);
              pw[TERMS - 1][t][h][e] = turn(pack_bf16x2(p0 - bf16_lo(hi2), p1 - bf16_hi(hi2)));
            } else {
              pw[0][t][h][e] = turn(pack_f16x2(exp2_fast(x0 + lv[t][e] - wbase[0]), exp2_fast(x1 + lv[t][e] - wbase[1])));
            }
          }
      }

      // ---- weighted values: [16 dims] x [heads]
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint32_t v32 = st32 + t * tile_bytes + v_row;
        if (TYPE == LORA_KV_BF16) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            if (ANY && b >= nb) continue;
            uint32_t v[4];
            ldsm4t(v, v32 + (((2 * b + v_c) ^ sw) << 4));
#pragma unroll
            for (int h = 0; h < NT; ++h) {
              mma16816(o[h][b], v[0], v[1], v[2], v[3], pw[0][t][h][0], pw[0][t][h][1]);
              mma16816(o[h][b], v[0], v[1], v[2], v[3], pw[TERMS - 1][t][h][0], pw[TERMS - 1][t][h][1]);
            }
          }
        } else {
#pragma unroll
          for (int p = 0; p < (NB + 1) / 2; ++p) {
            if (ANY && 2 * p >= nb) continue;
            uint32_t w[4];
            ldsm4t(w, v32 + (((2 * p + v_c) ^ sw) << 4));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int b = 2 * p + x;
              if (b >= NB || (ANY && b >= nb)) continue;
              uint32_t v0, v1, v2, v3;  // even and odd dims of tokens 0-7, then of 8-15
              codes_to_f16<TYPE>(w[2 * x], v0, v1);
              codes_to_f16<TYPE>(w[2 * x + 1], v2, v3);
#pragma unroll
              for (int h = 0; h < NT; ++h) mma_f16(o[h][b], v0, v1, v2, v3, pw[0][t][h][0], pw[0][t][h][1]);
            }
          }
        }
      }
      __syncwarp();  // (all lanes have read the stage)
      if (++stage == a.n_stages) {
        stage = 0;
        phase ^= 1;
      }
    }
  }
  __syncthreads();

  // ---- join what the warps' borders cut: pieces of one unit follow one another
  const bool broken = dead_block != 0;
  if (warp == 0) {
    const int4 p = lane < 2 * n_warps ? piece[lane] : make_int4(-1, 0, 0, 0);
    const unsigned there = __ballot_sync(~0u, p.x >= 0), below = there & ((1u << lane) - 1u);
    const int prev = below ? 31 - __clz(below) : lane;
    const int px = __shfl_sync(~0u, p.x, prev), pu = __shfl_sync(~0u, p.y, prev);
    const bool first = p.x >= 0 && (!below || px != p.x || pu != p.y);
    const unsigned firsts = __ballot_sync(~0u, first);
    if (p.x >= 0) order[__popc(below)] = lane;
    if (first) run[__popc(firsts & ((1u << lane) - 1u))] = __popc(below);
    if (lane == 0) {
      n_runs = __popc(firsts);
      run[__popc(firsts)] = __popc(there);
    }
  }
  // Meanwhile a thread each for the unit this block begins in (warp 1) and the
  // one it ends in (2): whether the block's border cuts it, into which blocks, and
  // a first look at their counter.
  int cut_first = 0, cut_count = 0;
  unsigned long long cut_seen = 0;
  if ((warp == 1 || warp == 2) && lane == 0) {
    const int which = warp - 1;
    to_join[which] = make_int2(0, 0);
    if (slots > 0) {
      const int at = which ? n_warps : 0;
      const int n = unit_slots(start[at].y, a.window, TT);
      const int in = (int)(from[at] - quotient(from[at], n) * n);  // slot of its unit
      // the unit's first and last step's slots in the list
      const long long here = which ? b0 + slots - 1 : b0, s_first = here - in + 1, s_last = here - in + n - 1;
      if (which ? in > 0 && s_last > here && s_first >= b0 : in > 1) {
        auto block_of = [&](unsigned long long slot) {
          const unsigned long long big = (each + 1) * more;
          return (int)(slot < big ? quotient(slot, each + 1) : more + quotient(slot - big, each));
        };
        cut_first = block_of(s_first);
        cut_count = block_of(s_last) - cut_first + 1;
        cut_seen = __ldcg(a.done + cut_first);
      }
    }
  }
  __syncthreads();
  // a thread has 8 dims of a row
  const int octs = dim / 8;
  const int per_run = a.rows * octs;
#pragma unroll 1
  for (int i0 = tid; i0 < n_runs * per_run && !broken; i0 += blockDim.x) {
    const int k = i0 / per_run, r = (i0 - k * per_run) / octs, d = (i0 - k * per_run - r * octs) * 8;
    const int f = run[k], e = run[k + 1];
    const int4 p0 = piece[order[f]], p1 = piece[order[e - 1]];
    const bool whole = !(p0.z & 1) && !(p1.z & 2);
    const int kvh = unit_kvh(p0.y), h0 = unit_h0(p0.y);
    if (h0 + r >= a.group) continue;
    Joined x;
    x.add<2, false>(f, e, 1, [&](int i) { return where[order[i]]; }, r, a.rows, state_head(a.rows) + r * dim + d);
    if (whole) {
      const int hd = kvh * a.group + h0 + r;
      const Ends fin = finish(a.sinks, hd, x.m, x.l);
      if (a.lse && d == 0) a.lse[(long long)p0.x * a.n_heads + hd] = fin.lse;
      store8(a.out + p0.x * a.ldo + ((long long)hd * dim + d) * 2, x.y, fin.mul);
    } else {
      float *st = a.part + ((size_t)blockIdx.x * 2 + (p0.z & 1 ? 0 : 1)) * floats;
      if (d == 0) {
        st[r] = x.m;
        st[a.rows + r] = x.l;
      }
      float4 *to = reinterpret_cast<float4 *>(st + state_head(a.rows) + r * dim + d);
      to[0] = make_float4(x.y[0], x.y[1], x.y[2], x.y[3]);
      to[1] = make_float4(x.y[4], x.y[5], x.y[6], x.y[7]);
    }
  }
  __syncthreads();

  // ---- count this block in for the units its borders cut; the last of a unit's blocks joins
  if (cut_count) {
    if (broken)  // (no result for what this block was to add to)
#pragma unroll 1
      for (int r = 0; r < a.rows; ++r) a.part[((size_t)blockIdx.x * 2 + warp - 1) * floats + a.rows + r] = -1.f;
    __threadfence();
    unsigned long long next;
    do {
      next = (cut_seen >> kCountBits) == a.tag ? cut_seen + 1 : a.tag << kCountBits | 1;
      const unsigned long long was = atomicCAS(a.done + cut_first, cut_seen, next);
      if (was == cut_seen) break;
      cut_seen = was;
    } while (true);
    __threadfence();
    if ((int)(next & ((1u << kCountBits) - 1u)) == cut_count) {
      a.done[cut_first] = 0;
      to_join[warp - 1] = make_int2(cut_first, cut_count);
    }
  }
  __syncthreads();
  if (to_join[0].y + to_join[1].y) {
    // Both units' rows by all threads, 8 dims of a row each; where they are fewer
    // than the threads the parts are shared out among groups of them.
    int seq[2], kvh[2], h0[2], items[2];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const int at = which ? n_warps : 0;
      items[which] = 0;
      if (!to_join[which].y) continue;
      const int un = (int)quotient(from[at], unit_slots(start[at].y, a.window, TT));
      seq[which] = start[at].x;
      kvh[which] = un / a.head_groups;
      h0[which] = (un - kvh[which] * a.head_groups) * ROWS;
      items[which] = min(a.rows, a.group - h0[which]) * octs;
    }
    const int all = items[0] + items[1];
    const int groups = max(1, min((int)blockDim.x / all, max(to_join[0].y, to_join[1].y)));
    Joined *share = reinterpret_cast<Joined *>(smem);  // (the rings are idle)
    auto put = [&](const Joined &x, int which, int r, int d) {
      if (x.gone) return;  // (the row stays as it was)
      const int hd = (which ? kvh[1] : kvh[0]) * a.group + (which ? h0[1] : h0[0]) + r;
      const long long row = which ? seq[1] : seq[0];
      const Ends e = finish(a.sinks, hd, x.m, x.l);
      if (a.lse && d == 0) a.lse[row * a.n_heads + hd] = e.lse;
      store8(a.out + row * a.ldo + ((long long)hd * dim + d) * 2, x.y, e.mul);
    };
#pragma unroll 1
    for (int i = tid; i < all * groups; i += blockDim.x) {
      const int grp = i / all, which = i - grp * all >= items[0], at = i - grp * all - (which ? items[0] : 0);
      const int r = at / octs, d = (at - r * octs) * 8;
      const int2 job = to_join[which];
      // the first block's own part (1), then those after it (0)
      auto state = [&](int k) { return a.part + ((size_t)(job.x + k) * 2 + (k ? 0 : 1)) * floats; };
      Joined x;
      x.add<4, true>(grp, job.y, groups, state, r, a.rows, state_head(a.rows) + r * dim + d);
      if (groups == 1)
        put(x, which, r, d);
      else
        share[i] = x;
    }
    if (groups > 1) {
      __syncthreads();
      if (tid < all) {
        const int which = tid >= items[0], at = tid - (which ? items[0] : 0), r = at / octs;
        Joined x;
#pragma unroll 1
        for (int k = 0; k < groups; ++k) {  // (a group without a part has the empty state)
          const Joined &z = share[k * all + tid];
          const float top = fmaxf(x.m, z.m), base = top == -INFINITY ? 0.f : top;
          const float u = exp2_fast(x.m - base), w = exp2_fast(z.m - base);
          x.m = top;
          x.l = fmaf(w, z.l, x.l * u);
          x.gone |= z.gone;
#pragma unroll
          for (int e = 0; e < 8; ++e) x.y[e] = fmaf(w, z.y[e], x.y[e] * u);
        }
        put(x, which, r, (at - r * octs) * 8);
      }
    }
  }

  // ---- sequences without a token: zeros, or untouched (length -1, and lengths in error)
#pragma unroll 1
  for (int i0 = blockIdx.x + warp * 32 * gridDim.x; i0 < s.n; i0 += gridDim.x * blockDim.x) {
    const int i = i0 + lane * gridDim.x;
    int len = 1;
    if (i < s.n) {
      len = __ldg(s.lens + i);
      if (len < -1 || !kv_len_ok(kv, s, len)) set_status(kv.status, LORA_ERR_BAD_ID);
    }
    unsigned empty = __ballot_sync(~0u, len == 0);
    while (empty) {
      const int z = __ffs(empty) - 1;
      empty &= empty - 1;
      const int q = i0 + z * gridDim.x;
#pragma unroll 1
      for (int c = lane; c < a.n_heads * dim / 8; c += 32)
        *reinterpret_cast<uint4 *>(a.out + q * a.ldo + c * 16) = make_uint4(0, 0, 0, 0);
      if (a.lse)
#pragma unroll 1
        for (int h = lane; h < a.n_heads; h += 32)
          a.lse[(long long)q * a.n_heads + h] = a.sinks ? a.sinks[h] : -INFINITY;
    }
  }
}

// ------------------------------------------------------------------ variants

using AttendKernel = void (*)(KvView, KvSeqs, AttendArgs);

// Which kernel takes a cache and a number of heads:
//  - a step has as many tiles as give it about 8 KiB, so that its own cost (a
//    wait, the running maximum) is spread over as many bytes: one tile instead of
//    two took 121 instead of 111 us for 512 requests of e4m3, 32 / 8 heads of 128;
//  - 12 warps where their registers suffice (up to 8 heads a unit, dims up to 128):
//    64 requests of bf16, 32 heads of 128, 182.5 us, with 8 warps 190; 512 of e4m3 111
//    and 117; 8 where accumulators would spill: 512 of e4m3, 64 / 4 heads of 128, 95 us,
//    with 12 warps 127.  (9 to 16 heads wider than 128 spill 50 to 260 bytes all the same:
//    a warp's 16 x 256 sums and as many of q are more than its registers.)
//  - the usual widths are constants, others take the loops of the next larger one
//    with a test for each 16 dims.
struct Variant {
  AttendKernel kernel[2];  // up to 8 query heads per key head, more
  int tt, warps[2];
};

// One file per cache type, so that they compile side by side.
Variant attend_variant_bf16(int dim);
Variant attend_variant_e4m3(int dim);
Variant attend_variant_int8(int dim);

template <int TYPE, int DIM, bool ANY, int TT, int WARPS>
Variant variant() {
  return {{attend_kernel<TYPE, DIM, ANY, TT, WARPS, 1>, attend_kernel<TYPE, DIM, ANY, TT, 8, 2>}, TT, {WARPS, 8}};
}

template <int TYPE>
Variant variant_of(int dim) {
  constexpr int W = TYPE == LORA_KV_BF16 ? 1 : 2;
  if (dim == 64) return variant<TYPE, 64, false, 2 * W, 12>();
  if (dim == 128) return variant<TYPE, 128, false, W, 12>();
  if (dim == 256) return variant<TYPE, 256, false, 1, 8>();
  return dim < 128 ? variant<TYPE, 128, true, W, 12>() : variant<TYPE, 256, true, 1, 8>();
}

}  // namespace lora
