// attend.cu -- attention of one new token per sequence over the paged cache.
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
// heads to a byte.  So the split is by bytes, evenly, whatever the lengths:
//  - The batch is one flat list of steps, ordered by (sequence, unit, step).  A
//    unit is one key head with up to 8 (or 16) of its query heads; a step is 16
//    TT consecutive tokens of it.  Each block takes an equal range of the list
//    (one block per SM), each of its warps an equal range of the block's.  Every
//    block finds its place itself from the lengths (one scan), so there is no
//    plan to keep and nothing of it is read on the host.
//  - A warp is on its own: one lane fetches its steps' tiles with bulk copies
//    (one per 16 tokens: a tile is contiguous in the cache, K, V and scales)
//    into the warp's ring of stages, several steps ahead, through the page
//    table; there is no block-wide synchronisation until the end.
//  - A (sequence, unit) that lies inside one warp's range is written at once.
//    States of ranges that cut one are joined in the block, in token order;
//    what a block's border cuts goes to the workspace and is joined by a second,
//    small launch (again in order: equal inputs give equal bits).
//
// The products run on the warp-level tensor instruction (m16n8k16, bf16): a
// unit's 8 query heads are few rows, and tcgen05 takes no fewer than 64.  With
// at most 8 heads the 16 rows carry each head twice; for the scores both copies
// give the same number, and for the values the first copy multiplies the bf16
// rounding of the weights and the second what the rounding left, so that the
// weights keep about 16 bits at no further instruction (rounded weights alone
// would add an error of the size of the result's own rounding).  With 9 to 16
// heads the rows are all different and the rest is a second instruction.
// 8-bit codes become bf16 exactly, with integer instructions on four at a time;
// the scales of K multiply the scores, those of V the weights, in fp32.
//
// Tokens outside the range get weight 0 by selection, not by adding: what lies
// in their places (the end of a page, before the window) may be anything.
#include "kv.cuh"

namespace lora {

constexpr int kAttMaxWarps = 8;
constexpr int kAttMaxStages = 8;
constexpr int kAttSmem = 227 * 1024;
constexpr int kJoinThreads = 512;

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
  // workspace: what each block's borders cut
  int4 *cut;           // [blocks] {sequence (-1: none), unit, last block, 0}: a unit that starts in the block and goes on
  float *part;         // [blocks][2] states: 0 continues from the block before, 1 starts here
  float *first;        // [blocks][warps] states: a warp's first piece, when more of its range follows,
  int first_in_smem;   // or where in shared memory those are (0: not there)
};

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

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
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

// How the scores of a unit are formed.
//  kBf16: q as it is, times bf16 keys.
//  kE4m3: q (scaled per head by a power of two to at most 256) as hi + lo / 32, both
//         e4m3: exact down to 2^-14 of the head's largest |q|, below that off by at
//         most 2^-23 of it.  Keys are multiplied as the codes they are.
//  kInt8: q = (hi + lo / 128 + rest / 16384) * amax / 127, all int8: off by at most
//         2^-22 of the largest |q|.  Products and sums are exact.
//  kF16:  q scaled by a power of two to fp16 (as exact as kE4m3), int8 keys as
//         fp16; with 9 to 16 heads, where three products of int8 would take more
//         registers than there are.
// hi and lo of the two 8-bit forms share an instruction while a unit has at
// most 8 heads: rows 0-7 are hi, rows 8-15 lo.
enum { kBf16, kE4m3, kInt8, kF16 };
__host__ __device__ constexpr int score_form(int type, bool wide) {
  return type == LORA_KV_BF16 ? kBf16 : type == LORA_KV_E4M3 ? kE4m3 : wide ? kF16 : kInt8;
}
__host__ __device__ constexpr int q_regs(int form, int nb, bool wide) {
  const int pairs = (nb + 1) / 2;
  return form == kE4m3 ? pairs * (wide ? 8 : 4) : form == kInt8 ? pairs * 6 : nb * (wide ? 4 : 2);
}

// Length of sequence s where it is one that is attended to, else 0 (none, empty, in error).
__device__ __forceinline__ int seq_len(const KvView &kv, const KvSeqs &s, int i) {
  const int len = __ldg(s.lens + i);
  return len > 0 && len <= ((long long)s.max_pages << kv.log2_page) ? len : 0;
}
__device__ __forceinline__ int first_token(int len, int window) { return window && len > window ? len - window : 0; }
// Steps of a unit of a sequence: its tiles from the first token's to the last one's.
__device__ __forceinline__ int seq_steps(int len, int window, int tt) {
  const int tiles = (len + kTileTokens - 1) / kTileTokens - first_token(len, window) / kTileTokens;
  return (tiles + tt - 1) / tt;
}

// Write row r's result from its state: o = sums for 4 dims, m and l over all tokens.
struct Ends {
  float mul, lse;
};
__device__ __forceinline__ Ends finish(const AttendArgs &a, int head, float m, float l) {
  Ends e;
  float base = m;
  if (a.sinks) {
    const float sink = a.sinks[head] * 1.44269504f;
    base = fmaxf(m, sink);
    l = l * exp2_fast(m - base) + exp2_fast(sink - base);
  }
  e.mul = __fdividef(exp2_fast(m - base), l);
  if (m == -INFINITY && !a.sinks) e.mul = __int_as_float(0x7fc00000);  // (every score minus infinity: 0 / 0)
  e.lse = fmaf(base, 0.693147181f, logf(l));
  return e;
}

// ------------------------------------------------------------------ kernel

// What a stage of a ring holds.
struct Step {
  int seq, unit, pos, len;  // sequence, unit, first token of the step, tokens of the sequence
};

// DIM: the head's width, or with ANY the largest of a range of multiples of 16 (kv.dim is the width).
// TT: tiles of 16 tokens per step.  WIDE: 9..16 query heads to a unit (else up to 8).
template <int TYPE, int DIM, bool ANY, int TT, bool WIDE>
__global__ void __launch_bounds__(kAttMaxWarps * 32, 1) attend_kernel(KvView kv, KvSeqs s, AttendArgs a) {
  constexpr int ES = kv_elt(TYPE);
  constexpr int ROWS = WIDE ? 16 : 8;   // query heads of a unit
  constexpr int HALVES = WIDE ? 2 : 1;  // of which a thread has one or two
  constexpr int NB = DIM / 16;          // blocks of 16 dims
  const int dim = ANY ? kv.dim : DIM, nb = ANY ? kv.dim / 16 : NB;
  const int row_bytes = dim * ES, chunks = row_bytes / 16;
  const int tile_bytes = kv_tile_bytes(TYPE, dim), stage_bytes = TT * tile_bytes;

  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kAttMaxWarps][kAttMaxStages];
  __shared__ Step held[kAttMaxWarps][kAttMaxStages];
  __shared__ int bad_tiles[kAttMaxWarps][kAttMaxStages];  // bit i: tile i of the stage is on no page of the cache
  __shared__ long long scan[kAttMaxWarps], from[kAttMaxWarps];  // from: a warp's first step, from its sequence's first
  __shared__ int2 start[kAttMaxWarps];                          // {sequence, length} of it
  __shared__ int4 piece[2 * kAttMaxWarps];  // [2 warp + which]: {sequence (-1: none), unit, cut before 1 / after 2, -}
  __shared__ const float *where[2 * kAttMaxWarps];
  __shared__ int order[2 * kAttMaxWarps], run[2 * kAttMaxWarps + 1];  // pieces in order; where each unit's run starts
  __shared__ int n_runs, dead_block, tail_steps;  // tail_steps: of the unit that the block's end cuts, behind it

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
  long long mine = 0;
  for (int i = s0; i < s1; ++i) mine += seq_steps(seq_len(kv, s, i), a.window, TT);
  long long before = mine;  // inclusive scan over the block
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(~0u, before, d);
    if (lane >= d) before += x;
  }
  if (lane == 31) scan[warp] = before;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int i = 0; i < kAttMaxWarps; ++i)
    if (i < n_warps) {
      if (i < warp) before += scan[i];
      total += scan[i];
    }
  before -= mine;
  // (no more blocks than steps: the join counts on every block in a row having a part)
  const unsigned long long steps_all = (unsigned long long)total * a.units;
  const unsigned blocks = (unsigned)min((unsigned long long)gridDim.x, steps_all);
  unsigned long long each = 0;  // steps of a block; the first `more` have one more
  unsigned more = 0;
  if (steps_all >> 32)
    each = steps_all / max(blocks, 1u);
  else
    each = (unsigned)steps_all / max(blocks, 1u);
  more = (unsigned)(steps_all - each * blocks);
  const long long b0 = each * blockIdx.x + min(blockIdx.x, more);
  const int steps = blockIdx.x < blocks ? (int)each + (blockIdx.x < more) : 0;
  const int wq = steps / n_warps, wr = steps - wq * n_warps;
  if (mine > 0) {  // whose range starts in this thread's sequences
    const long long lo = before * a.units - b0, hi = lo + mine * a.units;
    if (lo < steps && hi > 0) {
      for (int w = 0; w < n_warps; ++w) {
        const int at = wq * w + min(w, wr);
        if (at < lo || at >= hi || at >= steps) continue;
        long long p = lo;
        for (int i = s0; i < s1; ++i) {
          const int len = seq_len(kv, s, i);
          const long long e = p + (long long)seq_steps(len, a.window, TT) * a.units;
          if (at < e) {
            start[w] = make_int2(i, len);
            from[w] = at - p;
            break;
          }
          p = e;
        }
      }
    }
  }
  __syncthreads();
  const int count = wq + (warp < wr);  // this warp's steps

  uint8_t *ring = smem + (size_t)warp * a.n_stages * stage_bytes;
  if (count > 0) {
    // ---- fetching side: the next step to fetch, and pages of up to 32 tiles
    int left = count;  // steps not yet fetched
    int fseq = start[warp].x, flen = start[warp].y;
    int fsteps = seq_steps(flen, a.window, TT), ft0 = first_token(flen, a.window) / kTileTokens;
    int funit, fstep;
    {
      const unsigned long long off = from[warp];
      if (off >> 32) {
        funit = (int)(off / (unsigned)fsteps);
        fstep = (int)(off - (unsigned long long)funit * fsteps);
      } else {
        funit = (int)((unsigned)off / (unsigned)fsteps);
        fstep = (int)((unsigned)off - (unsigned)funit * fsteps);
      }
    }
    const bool starts_inside = fstep != 0;  // of its unit
    const long long head_stride = kv_head_stride(kv);
    const uint8_t *fhead = kv.base + (funit / a.head_groups) * head_stride;
    int pages = 0, pbase = -1;  // lane j: page of the sequence's tile pbase + j

    auto fetch = [&](int stage) {
      if (left <= 0) return;
      --left;
      const int tiles = (flen + kTileTokens - 1) / kTileTokens;
      const int t = ft0 + fstep * TT, want = ft0 + (fstep * TT & ~31);
      if (want != pbase) {
        pbase = want;
        pages = -1;
        if (pbase + lane < tiles)
          pages = __ldg(s.table + (long long)fseq * s.max_pages + (((pbase + lane) * kTileTokens) >> kv.log2_page));
      }
      // lane i fetches tile t + i
      const int page = TT == 1 ? __shfl_sync(~0u, pages, t - pbase) : __shfl_sync(~0u, pages, (t - pbase + lane) & 31);
      const bool wanted = lane < TT && t + lane < tiles;
      const long long at = wanted ? kv_tile_offset(kv, page, (t + lane) * kTileTokens) : -1;
      const unsigned ok = __ballot_sync(~0u, at >= 0), need = __ballot_sync(~0u, wanted);
      if (lane == 0) {
        held[warp][stage] = {fseq, funit, t * kTileTokens, flen};
        bad_tiles[warp][stage] = need & ~ok;
        mbar_arrive_expect_tx(&full[warp][stage], __popc(ok) * tile_bytes);
        if (need & ~ok) set_status(kv.status, LORA_ERR_BAD_ID);
      }
      __syncwarp();
      if (at >= 0) bulk_g2s(ring + stage * stage_bytes + lane * tile_bytes, fhead + at, tile_bytes, &full[warp][stage]);
      if (++fstep == fsteps) {
        fstep = 0;
        if (++funit == a.units) {
          funit = 0;
          pbase = -1;
          if (left > 0) {
            do {
              ++fseq;
              flen = seq_len(kv, s, fseq);
            } while (flen == 0);
            fsteps = seq_steps(flen, a.window, TT);
            ft0 = first_token(flen, a.window) / kTileTokens;
          }
        }
        fhead = kv.base + (funit / a.head_groups) * head_stride;
      }
    };

    // ---- computing side
    const uint32_t ring32 = smem_u32(ring);
    const int row = lane >> 2, quad = lane & 3;
    const int r8 = lane & 7, mat = lane >> 3;  // this lane's row and matrix of an ldmatrix
    const int low = chunks & -chunks, grp = low < 8 ? low : 8;
    const int sw = (r8 / (8 / grp)) & (grp - 1);  // its rows' chunk permutation (rows r8 and r8 + 8 share it)
    // K: bf16 (tokens 0-7 | 8-15) x (dims 0-7 | 8-15); 8-bit (tokens) x (dim blocks 2i | 2i + 1).  V: transposed.
    const uint32_t k_row = ((TYPE == LORA_KV_BF16 ? mat >> 1 : mat & 1) * 8 + r8) * row_bytes;
    const int k_c = TYPE == LORA_KV_BF16 ? mat & 1 : mat >> 1;
    const uint32_t v_row = (kTileTokens + (mat & 1) * 8 + r8) * row_bytes;
    const int v_c = mat >> 1;

    constexpr int FORM = score_form(TYPE, WIDE);
    uint32_t qa[q_regs(FORM, NB, WIDE)];
    float qs[HALVES];  // what a score is multiplied by for q's scaling
    float o[2 * NB][4], m[HALVES], l[HALVES], vtop = 0.f;  // vtop: largest V scale so far (8 bits)
    int cseq = -1, cunit = -1;
    bool cut_before = false;
    int stage = 0, fstage = 0;
    uint32_t phase = 0;

    // q as the products' A operand: rows = heads, columns = dims in the order of the K operand
    auto load_q = [&]() {
      const int kvh = cunit / a.head_groups, h0 = (cunit - kvh * a.head_groups) * ROWS;
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        const bool live = h0 + row + 8 * h < a.group;
        const uint8_t *q = a.q + cseq * a.ldq + (long long)(kvh * a.group + h0 + row + 8 * h) * dim * 2;
        uint2 u[NB];  // bf16: dims 16 b + 2 quad, + 1, + 8, + 9; 8 bits: dims 16 b + 4 quad ..
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          u[b] = make_uint2(0, 0);
          if (!live || (ANY && b >= nb)) continue;
          if (TYPE == LORA_KV_BF16) {
            u[b].x = __ldg(reinterpret_cast<const uint32_t *>(q + b * 32 + quad * 4));
            u[b].y = __ldg(reinterpret_cast<const uint32_t *>(q + b * 32 + quad * 4 + 16));
          } else {
            u[b] = __ldg(reinterpret_cast<const uint2 *>(q + b * 32 + quad * 8));
          }
        }
        if (FORM == kBf16) {
          qs[h] = 1.f;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            qa[b * 2 * HALVES + h] = u[b].x;
            qa[b * 2 * HALVES + HALVES + h] = u[b].y;
          }
          continue;
        }
        uint32_t top = 0;  // bits of the head's largest |q|
#pragma unroll
        for (int b = 0; b < NB; ++b)
          top = max(top, max(max(u[b].x & 0x7fffu, (u[b].x >> 16) & 0x7fffu), max(u[b].y & 0x7fffu, (u[b].y >> 16) & 0x7fffu)));
        top = max(top, __shfl_xor_sync(~0u, top, 1));
        top = max(top, __shfl_xor_sync(~0u, top, 2));
        const float amax = fmaxf(__uint_as_float(top << 16), 0x1p-100f);  // (a NaN is lost here and comes back below)
        const float nan = top >= 0x7f80u ? __int_as_float(0x7fc00000) : 0.f;
        const float two = __uint_as_float(__float_as_uint(amax) & 0x7f800000u);  // 2^E, 2^E <= amax
        if (FORM == kE4m3) {
          const float mul = 0x1p7f / two;
          qs[h] = two * 0x1p-7f + nan;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const float x[4] = {bf16_lo(u[b].x) * mul, bf16_hi(u[b].x) * mul, bf16_lo(u[b].y) * mul, bf16_hi(u[b].y) * mul};
            const uint32_t hi = e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16;
            float y[4];
            decode4<LORA_KV_E4M3>(hi, y);
            const uint32_t lo = e4m3x2((x[0] - y[0]) * 32.f, (x[1] - y[1]) * 32.f) |
                                e4m3x2((x[2] - y[2]) * 32.f, (x[3] - y[3]) * 32.f) << 16;
            const int k = (b >> 1) * 4 * HALVES + (b & 1) * 2;  // a0, a1 | a2, a3 of a pair of blocks
            if (WIDE) {
              qa[k + h] = hi;
              qa[k + 4 + h] = lo;
            } else {
              qa[k] = hi;
              qa[k + 1] = lo;
            }
          }
          if (NB & 1) qa[(NB / 2) * 4 * HALVES + 2] = qa[(NB / 2) * 4 * HALVES + 3] = 0;
        } else if (FORM == kInt8) {
          const float mul = 127.f / amax;
          qs[h] = amax * (1.f / (127.f * 16384.f)) + nan;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            float x[4] = {bf16_lo(u[b].x) * mul, bf16_hi(u[b].x) * mul, bf16_lo(u[b].y) * mul, bf16_hi(u[b].y) * mul};
            uint32_t t[3];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              t[k] = int8x4(x[0], x[1], x[2], x[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = (x[e] - (float)(int8_t)(t[k] >> (8 * e))) * 128.f;
            }
            const int k = (b >> 1) * 6 + (b & 1) * 2;
            qa[k] = t[0];
            qa[k + 1] = t[1];
            qa[(b >> 1) * 6 + 4 + (b & 1)] = t[2];
          }
        } else {  // kF16
          const float mul = 1.f / two;
          qs[h] = two + nan;
#pragma unroll
          for (int b = 0; b < NB; ++b) {  // even dims, then odd ones
            qa[b * 4 + h] = pack_f16x2(bf16_lo(u[b].x) * mul, bf16_lo(u[b].y) * mul);
            qa[b * 4 + 2 + h] = pack_f16x2(bf16_hi(u[b].x) * mul, bf16_hi(u[b].y) * mul);
          }
        }
      }
    };

    // (the first iterations fill the ring: one place in the code for each part)
    for (int i = 1 - a.n_stages;; ++i) {
      fetch(fstage);
      if (++fstage == a.n_stages) fstage = 0;
      if (i < 0) continue;
      const bool end = i == count;
      Step st = held[warp][stage];
      if (end || st.seq != cseq || st.unit != cunit) {
        if (cseq >= 0) {
          // The unit's state leaves the registers: as its result when the warp
          // has seen all of it, else as a piece to be joined.  At the range's
          // end the fetching side, just past it, tells whether the unit ends
          // too; the ring is then free for the state.
          const bool cut_after = end && fstep != 0;
          const bool whole = !cut_before && !cut_after;
          const int kvh = cunit / a.head_groups, h0 = (cunit - kvh * a.head_groups) * ROWS;
          float *state = end ? reinterpret_cast<float *>(ring) : a.first_in_smem
                             ? reinterpret_cast<float *>(smem + a.first_in_smem) + warp * floats
                             : a.first + ((size_t)blockIdx.x * kAttMaxWarps + warp) * floats;
          if (!whole && lane == 0) {
            const int k = 2 * warp + (cut_before ? 0 : 1);
            piece[k] = make_int4(cseq, cunit, (cut_before ? 1 : 0) | (cut_after ? 2 : 0), 0);
            where[k] = state;
            if (cut_after && warp == (wq ? n_warps : wr) - 1) tail_steps = fsteps - fstep;  // (the block's last steps)
          }
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            l[h] += __shfl_xor_sync(~0u, l[h], 1);
            l[h] += __shfl_xor_sync(~0u, l[h], 2);
            const int r = row + 8 * h, hd = kvh * a.group + h0 + r;
            if (r >= a.rows || h0 + r >= a.group) continue;
            float mul = TYPE == LORA_KV_BF16 ? 1.f : vtop * 0x1p-15f;
            uint8_t *out = a.out + cseq * a.ldo + (long long)hd * dim * 2;
            if (whole) {
              const Ends e = finish(a, hd, m[h], l[h]);
              mul *= e.mul;
              if (a.lse && quad == 0) a.lse[(long long)cseq * a.n_heads + hd] = e.lse;
            } else if (quad == 0) {
              state[r] = m[h];
              state[a.rows + r] = l[h];
            }
            float *sums = state + state_head(a.rows) + r * dim;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              if (ANY && b >= nb) continue;
              float x[4];  // n-tiles 2b and 2b + 1, columns 2 quad and 2 quad + 1
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float(&c)[4] = o[2 * b + (e >> 1)];
                x[e] = (WIDE ? c[(e & 1) + 2 * h] : c[e & 1] + c[(e & 1) + 2]) * mul;
              }
              if (TYPE == LORA_KV_BF16) {  // dims 16 b + 2 quad, + 1, + 8, + 9
                const int d = 16 * b + 2 * quad;
                if (whole) {
                  *reinterpret_cast<uint32_t *>(out + d * 2) = pack_bf16x2(x[0], x[1]);
                  *reinterpret_cast<uint32_t *>(out + d * 2 + 16) = pack_bf16x2(x[2], x[3]);
                } else {
                  *reinterpret_cast<float2 *>(sums + d) = make_float2(x[0], x[1]);
                  *reinterpret_cast<float2 *>(sums + d + 8) = make_float2(x[2], x[3]);
                }
              } else {  // n-tile 2b: even dims, 2b + 1: odd dims; 16 b + 4 quad ..
                const int d = 16 * b + 4 * quad;
                if (whole)
                  *reinterpret_cast<uint2 *>(out + d * 2) = make_uint2(pack_bf16x2(x[0], x[2]), pack_bf16x2(x[1], x[3]));
                else
                  *reinterpret_cast<float4 *>(sums + d) = make_float4(x[0], x[2], x[1], x[3]);
              }
            }
          }
        }
        if (end) break;
        cut_before = i == 0 && starts_inside;
        cseq = st.seq;
        cunit = st.unit;
#pragma unroll
        for (int h = 0; h < HALVES; ++h) m[h] = -INFINITY, l[h] = 0.f;
        vtop = 0.f;
#pragma unroll
        for (int n = 0; n < 2 * NB; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        load_q();
      }
      if (!mbar_wait_bounded(&full[warp][stage], phase, kv.status)) {
        // copies in flight must land before the block ends (again a bounded wait)
        for (int k = 0; k < a.n_stages; ++k) (void)mbar_wait_bounded(&full[warp][k], phase ^ (k < stage), kv.status);
        if (lane == 0) dead_block = 1;
        break;
      }
      const uint32_t st32 = ring32 + stage * stage_bytes;
      uint8_t *stp = ring + stage * stage_bytes;
      // tokens of the step that count: [lo, hi) of its 16 TT, without those on bad pages
      const int lo = first_token(st.len, a.window) - st.pos, hi = st.len - st.pos, bad = bad_tiles[warp][stage];
      const bool partial = lo > 0 || hi < kTileTokens * TT || bad;
      if (TYPE != LORA_KV_INT8 && partial) {
        // weight 0 times what lies there must be 0: clear V's rows outside (int8 has no NaN)
        for (int x = lane; x < kTileTokens * TT * chunks; x += 32) {
          const int t = x / chunks;
          if (t >= lo && t < hi && !(bad >> (t / kTileTokens) & 1)) continue;
          *reinterpret_cast<uint4 *>(stp + (t / kTileTokens) * tile_bytes + (kTileTokens + t % kTileTokens) * row_bytes +
                                     (x - t * chunks) * 16) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }

      // ---- scores: [heads] x [16 TT tokens]
      float c[2 * TT][4];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint32_t k32 = st32 + t * tile_bytes + k_row;
        float(&c0)[4] = c[2 * t], (&c1)[4] = c[2 * t + 1];
        float d0[4] = {}, d1[4] = {};  // a second sum: kE4m3's lo; kBf16's and kF16's odd blocks (a shorter chain)
        int i0[4] = {}, i1[4] = {}, r0[4] = {}, r1[4] = {};
        c0[0] = c0[1] = c0[2] = c0[3] = c1[0] = c1[1] = c1[2] = c1[3] = 0.f;
        if (FORM == kBf16) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            if (ANY && b >= nb) continue;
            uint32_t k[4];
            ldsm4(k, k32 + (((2 * b + k_c) ^ sw) << 4));
            const uint32_t *q = qa + b * 2 * HALVES;
            mma16816(b & 1 ? d0 : c0, q[0], q[HALVES - 1], q[HALVES], q[2 * HALVES - 1], k[0], k[1]);
            mma16816(b & 1 ? d1 : c1, q[0], q[HALVES - 1], q[HALVES], q[2 * HALVES - 1], k[2], k[3]);
          }
        } else {
#pragma unroll
          for (int p = 0; p < (NB + 1) / 2; ++p) {
            if (ANY && 2 * p >= nb) continue;
            uint32_t w[4];  // (tokens 0-7 | 8-15) x (block 2p | 2p + 1)
            ldsm4(w, k32 + (((2 * p + k_c) ^ sw) << 4));
            if ((ANY || (NB & 1)) && 2 * p + 1 >= nb) w[2] = w[3] = 0;  // (past the row's end: anything, NaN too)
            if (FORM == kE4m3) {
              const uint32_t *q = qa + p * 4 * HALVES;
              mma_e4m3(c0, q[0], q[1], q[2], q[3], w[0], w[2]);
              mma_e4m3(c1, q[0], q[1], q[2], q[3], w[1], w[3]);
              if (WIDE) {
                q += 4 * (HALVES - 1);
                mma_e4m3(d0, q[0], q[1], q[2], q[3], w[0], w[2]);
                mma_e4m3(d1, q[0], q[1], q[2], q[3], w[1], w[3]);
              }
            } else if (FORM == kInt8) {
              const uint32_t *q = qa + p * 6;
              mma_s8(i0, q[0], q[1], q[2], q[3], w[0], w[2]);
              mma_s8(i1, q[0], q[1], q[2], q[3], w[1], w[3]);
              mma_s8(r0, q[4], 0, q[5], 0, w[0], w[2]);
              mma_s8(r1, q[4], 0, q[5], 0, w[1], w[3]);
            } else {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int b = 2 * p + x;
                if (b >= NB || (ANY && b >= nb)) continue;
                const uint32_t *q = qa + b * 4;
                uint32_t even, odd;
                codes_to_f16<TYPE>(w[2 * x], even, odd);
                mma_f16(x ? d0 : c0, q[0], q[1], q[2], q[3], even, odd);
                codes_to_f16<TYPE>(w[2 * x + 1], even, odd);
                mma_f16(x ? d1 : c1, q[0], q[1], q[2], q[3], even, odd);
              }
            }
          }
        }
#pragma unroll
        for (int e = 0; e < (WIDE ? 4 : 2); ++e) {
          if (FORM == kE4m3) {
            c0[e] = fmaf(WIDE ? d0[e] : c0[(e + 2) & 3], 0.03125f, c0[e]);
            c1[e] = fmaf(WIDE ? d1[e] : c1[(e + 2) & 3], 0.03125f, c1[e]);
          } else if (FORM == kInt8) {
            c0[e] = fmaf((float)(i0[e] * 128 + i0[(e + 2) & 3]), 128.f, (float)r0[e]);
            c1[e] = fmaf((float)(i1[e] * 128 + i1[(e + 2) & 3]), 128.f, (float)r1[e]);
          } else {
            c0[e] += d0[e];
            c1[e] += d1[e];
          }
        }
      }

      // ---- weights
      float vs[2 * TT][2];
#pragma unroll
      for (int n = 0; n < 2 * TT; ++n) {
        const int t = n / 2, tok = (n & 1) * 8 + 2 * quad;  // of the tile
        float2 ks = make_float2(a.scale2, a.scale2);
        if (TYPE != LORA_KV_BF16) {
          const uint8_t *sc = stp + t * tile_bytes + 2 * kTileTokens * row_bytes;
          ks = *reinterpret_cast<const float2 *>(sc + tok * 4);
          ks.x *= a.scale2;
          ks.y *= a.scale2;
          const float2 u = *reinterpret_cast<const float2 *>(sc + (kTileTokens + tok) * 4);
          vs[n][0] = u.x;
          vs[n][1] = u.y;
        }
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          c[n][2 * h] *= FORM == kBf16 ? ks.x : ks.x * qs[h];
          c[n][2 * h + 1] *= FORM == kBf16 ? ks.y : ks.y * qs[h];
        }
        if (partial) {
          const bool off = bad >> t & 1;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = t * kTileTokens + tok + e;
            if (j < lo || j >= hi || off) {
              c[n][e] = c[n][2 + e] = -INFINITY;
              if (TYPE != LORA_KV_BF16) vs[n][e] = 0.f;
            }
          }
        }
      }
      float mx[HALVES], base_m[HALVES], fade = 1.f;
      bool moved = false;
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        mx[h] = m[h];
#pragma unroll
        for (int n = 0; n < 2 * TT; ++n) mx[h] = fmaxf(mx[h], fmaxf(c[n][2 * h], c[n][2 * h + 1]));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(~0u, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(~0u, mx[h], 2));
        base_m[h] = mx[h] == -INFINITY ? 0.f : mx[h];
        moved |= mx[h] > m[h];
      }
      float unit = 0.f;
      if (TYPE != LORA_KV_BF16) {
        // The weights times V's scales become fp16 in units of 2^-15 of the
        // largest scale so far: none overflows, and what is below 2^-29 of it
        // still has its place.
        float vm = vtop;
#pragma unroll
        for (int n = 0; n < 2 * TT; ++n) vm = fmaxf(vm, fmaxf(vs[n][0], vs[n][1]));
        vm = fmaxf(vm, __shfl_xor_sync(~0u, vm, 1));
        vm = fmaxf(vm, __shfl_xor_sync(~0u, vm, 2));
        if (vm > vtop) {
          fade = __fdividef(vtop, vm);
          vtop = vm;
          moved = true;
        }
        unit = vtop > 0.f ? 0x1p15f / vtop : 0.f;
      }
      if (__any_sync(~0u, moved)) {
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          float alpha = exp2_fast(m[h] - base_m[h]);
          l[h] *= alpha;
          m[h] = mx[h];
          alpha *= fade;
#pragma unroll
          for (int n = 0; n < 2 * NB; ++n) {
            if (ANY && n >= 2 * nb) continue;
            o[n][2 * h] *= alpha;
            o[n][2 * h + 1] *= alpha;
            if (!WIDE) {
              o[n][2] *= alpha;
              o[n][3] *= alpha;
            }
          }
        }
      }
      // as two terms: hi keeps the leading bits of the type (cut, so that the rest is exact), lo the rest's
      uint32_t ph[2 * TT][HALVES], pl[2 * TT][HALVES];
#pragma unroll
      for (int n = 0; n < 2 * TT; ++n)
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          float p0 = exp2_fast(c[n][2 * h] - base_m[h]), p1 = exp2_fast(c[n][2 * h + 1] - base_m[h]);
          l[h] += p0 + p1;
          if (TYPE == LORA_KV_BF16) {
            ph[n][h] = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
            pl[n][h] = pack_bf16x2(p0 - bf16_lo(ph[n][h]), p1 - bf16_hi(ph[n][h]));
          } else {
            p0 *= vs[n][0] * unit;
            p1 *= vs[n][1] * unit;
            const float h0 = __uint_as_float(__float_as_uint(p0) & 0xffffe000u);
            const float h1 = __uint_as_float(__float_as_uint(p1) & 0xffffe000u);
            ph[n][h] = pack_f16x2(h0, h1);
            pl[n][h] = pack_f16x2(p0 - h0, p1 - h1);
          }
        }

      // ---- weighted values
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint32_t v32 = st32 + t * tile_bytes + v_row;
        auto add = [&](float(&acc)[4], uint32_t b0, uint32_t b1) {
          auto mma = [&](uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
            if (TYPE == LORA_KV_BF16)
              mma16816(acc, a0, a1, a2, a3, b0, b1);
            else
              mma_f16(acc, a0, a1, a2, a3, b0, b1);
          };
          if (WIDE) {
            mma(ph[2 * t][0], ph[2 * t][HALVES - 1], ph[2 * t + 1][0], ph[2 * t + 1][HALVES - 1]);
            mma(pl[2 * t][0], pl[2 * t][HALVES - 1], pl[2 * t + 1][0], pl[2 * t + 1][HALVES - 1]);
          } else {
            mma(ph[2 * t][0], pl[2 * t][0], ph[2 * t + 1][0], pl[2 * t + 1][0]);
          }
        };
        if (TYPE == LORA_KV_BF16) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            if (ANY && b >= nb) continue;
            uint32_t v[4];
            ldsm4t(v, v32 + (((2 * b + v_c) ^ sw) << 4));
            add(o[2 * b], v[0], v[1]);
            add(o[2 * b + 1], v[2], v[3]);
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
              uint32_t e0, o0, e1, o1;
              codes_to_f16<TYPE>(w[2 * x], e0, o0);
              codes_to_f16<TYPE>(w[2 * x + 1], e1, o1);
              add(o[2 * b], e0, e1);
              add(o[2 * b + 1], o0, o1);
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
    // the last run goes on past the block and starts in it: the join finishes it, up to its last step's block
    int4 cut = make_int4(-1, 0, 0, 0);
    const int last_first = firsts ? 31 - __clz(firsts) : 0, last = there ? 31 - __clz(there) : 0;
    const int head_cut = __shfl_sync(~0u, p.z, last_first), tail_cut = __shfl_sync(~0u, p.z, last);
    cut.x = __shfl_sync(~0u, p.x, last);
    cut.y = __shfl_sync(~0u, p.y, last);
    if (!there || broken || !(tail_cut & 2) || (head_cut & 1)) {
      cut.x = -1;
    } else {
      const unsigned long long step = b0 + steps + tail_steps - 1, big = (each + 1) * more;
      cut.z = (int)(step < big ? step / (each + 1) : more + (step - big) / each);
    }
    if (lane == 0) a.cut[blockIdx.x] = cut;
  }
  if (broken && tid < 2 * a.rows)  // (no result for what this block was to add to)
    a.part[((size_t)blockIdx.x * 2 + tid / a.rows) * floats + a.rows + tid % a.rows] = -1.f;
  __syncthreads();
  const int quads = dim / 4;
  for (int k = 0; k < n_runs; ++k) {
    const int f = run[k], e = run[k + 1];
    const int4 p0 = piece[order[f]], p1 = piece[order[e - 1]];
    const bool whole = !(p0.z & 1) && !(p1.z & 2);
    const int kvh = p0.y / a.head_groups, h0 = (p0.y - kvh * a.head_groups) * ROWS;
    if (broken) break;
    for (int x = tid; x < a.rows * quads; x += blockDim.x) {
      const int r = x / quads, d = (x - r * quads) * 4;
      if (h0 + r >= a.group) break;
      float mm = -INFINITY, ll = 0.f;
      for (int i = f; i < e; ++i) mm = fmaxf(mm, where[order[i]][r]);
      const float bm = mm == -INFINITY ? 0.f : mm;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
      for (int i = f; i < e; ++i) {
        const float *st = where[order[i]];
        const float w = exp2_fast(st[r] - bm);
        const float4 z = *reinterpret_cast<const float4 *>(st + state_head(a.rows) + r * dim + d);
        ll = fmaf(w, st[a.rows + r], ll);
        y.x = fmaf(w, z.x, y.x);
        y.y = fmaf(w, z.y, y.y);
        y.z = fmaf(w, z.z, y.z);
        y.w = fmaf(w, z.w, y.w);
      }
      if (whole) {
        const int hd = kvh * a.group + h0 + r;
        const Ends fin = finish(a, hd, mm, ll);
        if (a.lse && d == 0) a.lse[(long long)p0.x * a.n_heads + hd] = fin.lse;
        *reinterpret_cast<uint2 *>(a.out + p0.x * a.ldo + ((long long)hd * dim + d) * 2) =
            make_uint2(pack_bf16x2(y.x * fin.mul, y.y * fin.mul), pack_bf16x2(y.z * fin.mul, y.w * fin.mul));
      } else {
        float *st = a.part + ((size_t)blockIdx.x * 2 + (p0.z & 1 ? 0 : 1)) * floats;
        if (d == 0) {
          st[r] = mm;
          st[a.rows + r] = ll;
        }
        *reinterpret_cast<float4 *>(st + state_head(a.rows) + r * dim + d) = y;
      }
    }
  }

  // ---- sequences without a token: zeros, or untouched (length -1, and lengths in error)
  for (int i0 = blockIdx.x + warp * 32 * gridDim.x; i0 < s.n; i0 += gridDim.x * blockDim.x) {
    const int i = i0 + lane * gridDim.x;
    int len = 1;
    if (i < s.n) {
      len = __ldg(s.lens + i);
      if (len < -1 || len > ((long long)s.max_pages << kv.log2_page)) set_status(kv.status, LORA_ERR_BAD_ID);
    }
    unsigned empty = __ballot_sync(~0u, len == 0);
    while (empty) {
      const int z = __ffs(empty) - 1;
      empty &= empty - 1;
      const int q = i0 + z * gridDim.x;
      for (int c = lane; c < a.n_heads * dim / 8; c += 32)
        *reinterpret_cast<uint4 *>(a.out + q * a.ldo + c * 16) = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (int h = lane; h < a.n_heads; h += 32)
          a.lse[(long long)q * a.n_heads + h] = a.sinks ? a.sinks[h] : -INFINITY;
    }
  }
}

// Joins the states of the units that a block's end cut: block b's own (part 1),
// then those of the blocks after it (part 0) up to the unit's last.  A thread
// has 4 dims of one head and every SPLITS-th state; the splits meet in shared
// memory.
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(AttendArgs a, int unit_rows, int dim) {
  __shared__ float sums[kJoinThreads * 4];
  __shared__ float tops[16], lens[kJoinThreads];
  __shared__ int broken;
  griddep_wait();
  griddep_launch_dependents();
  const int4 cut = a.cut[blockIdx.x];
  if (cut.x < 0) return;
  const int rows = a.rows, floats = state_floats(rows, dim), n = cut.z - blockIdx.x + 1;
  auto state = [&](int i) { return a.part + ((size_t)(blockIdx.x + i) * 2 + (i ? 0 : 1)) * floats; };
  const int h0 = (cut.y % a.head_groups) * unit_rows, live = min(rows, a.group - h0);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) broken = 0;
  __syncthreads();
  for (int r = warp; r < live; r += kJoinThreads / 32) {
    float mm = -INFINITY;
    bool bad = false;
    for (int i = lane; i < n; i += 32) {
      mm = fmaxf(mm, state(i)[r]);
      bad |= state(i)[rows + r] < 0.f;
    }
    for (int d = 16; d; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, d));
    if (__any_sync(~0u, bad) && lane == 0) broken = 1;
    if (lane == 0) tops[r] = mm;
  }
  __syncthreads();
  if (broken) return;
  const int per = dim / 4;                      // threads of a row
  const int at_once = max(1, kJoinThreads / per), splits = max(1, at_once / live);
  for (int r0 = 0; r0 < live; r0 += at_once) {  // (more than one pass only for 16 wide rows)
    const int slot = tid / per, d = (tid % per) * 4;
    const int r = r0 + slot / splits, sp = slot % splits;
    const bool on = slot < at_once && r < live;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    float ll = 0.f, mm = 0.f;
    if (on) {
      mm = tops[r];
      const float bm = mm == -INFINITY ? 0.f : mm;
#pragma unroll 4
      for (int i = sp; i < n; i += splits) {
        const float *st = state(i);
        const float w = exp2_fast(st[r] - bm);
        const float4 y = *reinterpret_cast<const float4 *>(st + state_head(rows) + r * dim + d);
        ll = fmaf(w, st[rows + r], ll);
        x.x = fmaf(w, y.x, x.x);
        x.y = fmaf(w, y.y, x.y);
        x.z = fmaf(w, y.z, x.z);
        x.w = fmaf(w, y.w, x.w);
      }
      *reinterpret_cast<float4 *>(sums + tid * 4) = x;
      lens[tid] = ll;
    }
    __syncthreads();
    if (on && sp == 0) {
      for (int k = 1; k < splits; ++k) {
        const float4 y = *reinterpret_cast<const float4 *>(sums + (tid + k * per) * 4);
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
        ll += lens[tid + k * per];
      }
      const int hd = (cut.y / a.head_groups) * a.group + h0 + r;
      const Ends e = finish(a, hd, mm, ll);
      if (a.lse && d == 0) a.lse[(long long)cut.x * a.n_heads + hd] = e.lse;
      *reinterpret_cast<uint2 *>(a.out + cut.x * a.ldo + ((long long)hd * dim + d) * 2) =
          make_uint2(pack_bf16x2(x.x * e.mul, x.y * e.mul), pack_bf16x2(x.z * e.mul, x.w * e.mul));
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host

namespace {

using AttendKernel = void (*)(KvView, KvSeqs, AttendArgs);

// Steps of about 8 KiB: several tiles where a tile is small, so that the cost
// of a step (a wait, the running maximum) is spread over as many bytes.
struct Variant {
  AttendKernel kernel[2];  // up to 8 query heads per key head, more
  int tt;
};

template <int TYPE, int DIM, bool ANY, int TT>
Variant variant() {
  return {{attend_kernel<TYPE, DIM, ANY, TT, false>, attend_kernel<TYPE, DIM, ANY, TT, true>}, TT};
}

template <int TYPE>
Variant variant_of(int dim) {
  constexpr int W = TYPE == LORA_KV_BF16 ? 1 : 2;
  if (dim == 64) return variant<TYPE, 64, false, 2 * W>();
  if (dim == 128) return variant<TYPE, 128, false, W>();
  if (dim == 256) return variant<TYPE, 256, false, 1>();
  return dim < 128 ? variant<TYPE, 128, true, W>() : variant<TYPE, 256, true, 1>();
}
Variant variant_of(int type, int dim) {
  return type == LORA_KV_BF16   ? variant_of<LORA_KV_BF16>(dim)
         : type == LORA_KV_E4M3 ? variant_of<LORA_KV_E4M3>(dim)
                                : variant_of<LORA_KV_INT8>(dim);
}

constexpr int kAttStatic = 2560;  // at least what the kernel's static shared memory takes

// Warps and stages: at least 3 stages a warp, 8 warps where that fits; the
// warps' first pieces (state_bytes each) stay in shared memory where that costs
// no warp.
struct Geometry {
  int warps, stages, first;  // first: its offset in dynamic shared memory (0: in the workspace)
  int smem;
};
Geometry geometry(int stage_bytes, int state_bytes) {
  const int room = kAttSmem - kAttStatic;
  Geometry g;
  g.warps = room / (3 * stage_bytes);
  g.warps = g.warps > kAttMaxWarps ? kAttMaxWarps : g.warps;
  const int keep = g.warps * state_bytes;
  const bool fits = room - keep >= 3 * stage_bytes * g.warps;
  g.stages = (room - (fits ? keep : 0)) / (g.warps * stage_bytes);
  g.stages = g.stages > kAttMaxStages ? kAttMaxStages : g.stages;
  g.first = fits ? g.warps * g.stages * stage_bytes : 0;
  g.smem = g.warps * g.stages * stage_bytes + (fits ? keep : 0);
  return g;
}

int group_of(const lora_kv *kv, int n_heads) { return n_heads / kv->heads; }

}  // namespace

int attend_setup(lora_kv *kv) {
  const Variant v = variant_of(kv->type, kv->dim);
  for (AttendKernel k : v.kernel) {
    const int rc = cuda_status(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttSmem - kAttStatic));
    if (rc != LORA_OK) return rc;
  }
  return LORA_OK;
}

size_t attend_workspace_bytes(const lora_kv *kv, int n_heads) {
  const int group = group_of(kv, n_heads);
  const size_t state = size_t(state_floats(group > 16 ? 16 : group, kv->dim)) * 4;
  return align256(size_t(kv->n_sm) * sizeof(int4)) + size_t(kv->n_sm) * (2 + kAttMaxWarps) * state;
}

int launch_attend(const lora_kv *kv, int layer, const KvSeqs &s, const AttendCall &c, cudaStream_t st) {
  const Variant v = variant_of(kv->type, kv->dim);
  AttendArgs a;
  a.q = static_cast<const uint8_t *>(c.q);
  a.out = static_cast<uint8_t *>(c.out);
  a.ldq = 2ll * c.ldq;
  a.ldo = 2ll * c.ldo;
  a.lse = c.lse;
  a.sinks = c.sinks;
  a.n_heads = c.n_heads;
  a.group = group_of(kv, c.n_heads);
  const bool wide = a.group > 8;
  const int unit_rows = wide ? 16 : 8;
  a.rows = a.group < unit_rows ? a.group : unit_rows;
  a.head_groups = (a.group + unit_rows - 1) / unit_rows;
  a.units = kv->heads * a.head_groups;
  a.scale2 = c.scale * 1.44269504f;
  a.window = c.window;
  const size_t floats = state_floats(a.rows, kv->dim);
  const Geometry g = geometry(v.tt * kv_tile_bytes(kv->type, kv->dim), int(floats * 4));
  a.n_stages = g.stages;
  a.first_in_smem = g.first;
  uint8_t *ws = static_cast<uint8_t *>(c.ws);
  a.cut = reinterpret_cast<int4 *>(ws);
  a.part = reinterpret_cast<float *>(ws + align256(size_t(kv->n_sm) * sizeof(int4)));
  a.first = a.part + size_t(kv->n_sm) * 2 * floats;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kv->n_sm);
  cfg.blockDim = dim3(g.warps * 32);
  cfg.dynamicSmemBytes = g.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0] = pdl_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int rc = cuda_status(cudaLaunchKernelEx(&cfg, v.kernel[wide], kv->view(layer), s, a));
  if (rc != LORA_OK) return rc;
  g_launches.fetch_add(1);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  rc = cuda_status(cudaLaunchKernelEx(&cfg, attend_join_kernel, a, unit_rows, kv->dim));
  if (rc == LORA_OK) g_launches.fetch_add(1);
  return rc;
}

}  // namespace lora
