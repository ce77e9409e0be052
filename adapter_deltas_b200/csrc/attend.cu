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
  float scale2;        // scale * log2(e)
  int window;
  int n_stages;
  // workspace: what each block's borders cut
  int4 *cut;           // [blocks] {sequence (-1: none), unit, last block, 0}: a unit that starts in the block and goes on
  float *part;         // [blocks][2] states: 0 continues from the block before, 1 starts here
  float *first;        // [blocks][warps] states: a warp's first range, when more follow
};

// A state in memory: m[rows], l[rows], then rows x dim weighted sums.
__host__ __device__ constexpr int state_floats(int rows, int dim) { return rows * (dim + 2); }

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

// Bytes 0 and 2 (even) and 1 and 3 (odd) of a word of codes as bf16 pairs, exactly.
//  e4m3: the exponent and mantissa bits moved to bf16's places are the value
//        times 2^-120 (the exponents' biases differ by 120), subnormals too.
//  int8: 128 + (code's low 7 bits) and 128 or 256 by its sign are bf16
//        numbers with the code's bits in place; their difference is the code.
template <int TYPE>
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t &even, uint32_t &odd) {
  const uint32_t v = w << 8;
  if (TYPE == LORA_KV_E4M3) {
    const uint32_t o = ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
    const uint32_t e = ((v >> 4) & 0x07f007f0u) | (v & 0x80008000u);
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(odd) : "r"(o), "r"(0x7b807b80u));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(even) : "r"(e), "r"(0x7b807b80u));
  } else {
    const uint32_t u = w >> 8;
    const uint32_t e0 = (w & 0x007f007fu) | 0x43004300u, e1 = (w & 0x00800080u) | 0x43004300u;
    const uint32_t o0 = (u & 0x007f007fu) | 0x43004300u, o1 = (u & 0x00800080u) | 0x43004300u;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(even) : "r"(e0), "r"(e1));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(odd) : "r"(o0), "r"(o1));
  }
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
  e.lse = (base + __log2f(l)) * 0.693147181f;
  return e;
}

// ------------------------------------------------------------------ kernel

// DIM: the head's width, or 256 for any multiple of 16 up to that (kv.dim).
// TT: tiles of 16 tokens per step.  WIDE: 9..16 query heads to a unit (else up to 8).
template <int TYPE, int DIM, int TT, bool WIDE>
__global__ void __launch_bounds__(kAttMaxWarps * 32, 1) attend_kernel(KvView kv, KvSeqs s, AttendArgs a) {
  constexpr int ES = kv_elt(TYPE);
  constexpr int ROWS = WIDE ? 16 : 8;   // query heads of a unit
  constexpr int NB = DIM / 16;          // blocks of 16 dims
  constexpr bool ANY = DIM == 256;
  const int dim = ANY ? kv.dim : DIM, nb = ANY ? kv.dim / 16 : NB;
  const int row_bytes = dim * ES, chunks = row_bytes / 16;
  const int tile_bytes = kv_tile_bytes(TYPE, dim), stage_bytes = TT * tile_bytes;

  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kAttMaxWarps][kAttMaxStages];
  __shared__ long long scan[kAttMaxWarps + 1];
  __shared__ int4 start[kAttMaxWarps];       // {sequence, unit, step, steps of the sequence}
  __shared__ int4 piece[kAttMaxWarps][2];    // {sequence, unit, state: cut before / after, 1 + where}
  __shared__ long long tail_end;             // flat end of the unit the block's end cuts
  __shared__ int list[2 * kAttMaxWarps], chain_of[2 * kAttMaxWarps];  // the pieces in order, and the unit's run of each
  __shared__ int n_pieces, n_chains;
  __shared__ int dead_block;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_warps = blockDim.x >> 5;
  const int floats = state_floats(ROWS, dim);

  if (lane < a.n_stages) mbar_init(&full[warp][lane], 1);
  fence_mbar_init();
  if (tid < 2 * kAttMaxWarps) piece[tid >> 1][tid & 1] = make_int4(-1, 0, 0, 0);
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
  long long total = 0, base = 0;
  for (int i = 0; i < n_warps; ++i) {
    if (i == warp) base = total;
    total += scan[i];
  }
  before += base - mine;
  const long long steps_all = total * a.units;
  // (no more blocks than steps: the join counts on every block in a row having a part)
  const long long blocks = min((long long)gridDim.x, steps_all);
  const long long b0 = blockIdx.x < blocks ? steps_all * blockIdx.x / blocks : 0;
  const long long b1 = blockIdx.x < blocks ? steps_all * (blockIdx.x + 1) / blocks : 0;
  if (mine > 0) {  // whose range starts in this thread's sequences
    const long long lo = before * a.units, hi = (before + mine) * a.units;
    for (int w = 0; w <= n_warps; ++w) {
      // (w == n_warps: the unit of the block's last step, for its end)
      const long long at = w < n_warps ? b0 + (b1 - b0) * w / n_warps : b1 - 1;
      const long long to = w < n_warps ? b0 + (b1 - b0) * (w + 1) / n_warps : b1;
      if (at >= to || at < lo || at >= hi || b0 >= b1) continue;
      long long p = lo;
      for (int i = s0; i < s1; ++i) {
        const int n = seq_steps(seq_len(kv, s, i), a.window, TT);
        const long long e = p + (long long)n * a.units;
        if (at < e) {
          const int unit = (int)((at - p) / n), step = (int)((at - p) % n);
          if (w < n_warps)
            start[w] = make_int4(i, unit, step, n);
          else
            tail_end = p + (long long)(unit + 1) * n;
          break;
        }
        p = e;
      }
    }
  }
  __syncthreads();
  const long long w0 = b0 + (b1 - b0) * warp / n_warps, w1 = b0 + (b1 - b0) * (warp + 1) / n_warps;

  uint8_t *ring = smem + (size_t)warp * a.n_stages * stage_bytes;
  const uint32_t ring32 = smem_u32(ring);
  bool dead = false;
  if (w0 < w1) {
    // ---- fetching side: the next step to fetch, and pages of up to 32 tiles
    long long left = w1 - w0;  // steps not yet fetched
    int fseq = start[warp].x, funit = start[warp].y, fstep = start[warp].z, fsteps = start[warp].w;
    int flen = seq_len(kv, s, fseq);
    int pages = 0, pbase = -1;  // lane j: page of the sequence's tile pbase + j
    int d_seq = 0, d_unit = 0, d_step = 0, d_len = 0, d_bad = 0;  // lane i: what stage i holds

    auto fetch = [&](int stage) {
      if (left <= 0) return;
      --left;
      const int t0 = first_token(flen, a.window) / kTileTokens, tiles = (flen + kTileTokens - 1) / kTileTokens;
      const int t = t0 + fstep * TT, want = t0 + (fstep * TT / 32) * 32;
      if (want != pbase) {
        pbase = want;
        pages = -1;
        if (pbase + lane < tiles)
          pages = __ldg(s.table + (long long)fseq * s.max_pages + (((pbase + lane) * kTileTokens) >> kv.log2_page));
      }
      const uint8_t *head = kv.base + (funit / a.head_groups) * kv_head_stride(kv);
      uint8_t *dst = ring + stage * stage_bytes;
      const uint8_t *src[TT];
      int n = 0, bad = 0;
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        src[i] = nullptr;
        const int page = __shfl_sync(~0u, pages, t + i - pbase);
        if (t + i < tiles) {
          const long long at = kv_tile_offset(kv, page, (t + i) * kTileTokens);
          if (at >= 0) {
            src[i] = head + at;
            ++n;
          } else {
            bad |= 1 << i;
          }
        }
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&full[warp][stage], n * tile_bytes);
#pragma unroll
        for (int i = 0; i < TT; ++i)
          if (src[i]) bulk_g2s(dst + i * tile_bytes, src[i], tile_bytes, &full[warp][stage]);
        if (bad) set_status(kv.status, LORA_ERR_BAD_ID);
      }
      if (lane == stage) {
        d_seq = fseq;
        d_unit = funit;
        d_step = fstep;
        d_len = flen;
        d_bad = bad;
      }
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
          }
        }
      }
    };
    for (int i = 0; i < a.n_stages; ++i) fetch(i);

    // ---- computing side
    const int row = lane >> 2, quad = lane & 3;
    const int r8 = lane & 7, mat = lane >> 3;  // this lane's row and matrix of an ldmatrix
    const int low = chunks & -chunks, grp = low < 8 ? low : 8;
    const int sw = (r8 / (8 / grp)) & (grp - 1);  // its rows' chunk permutation (rows r8 and r8 + 8 share it)
    // K: bf16 (tokens 0-7 | 8-15) x (dims 0-7 | 8-15); 8-bit (tokens) x (dim blocks 2i | 2i + 1).  V: transposed.
    const uint32_t k_row = ((TYPE == LORA_KV_BF16 ? mat >> 1 : mat & 1) * 8 + r8) * row_bytes;
    const int k_c = TYPE == LORA_KV_BF16 ? mat & 1 : mat >> 1;
    const uint32_t v_row = ((mat & 1) * 8 + r8) * row_bytes;
    const int v_c = mat >> 1;

    uint32_t qa[NB][WIDE ? 4 : 2];
    float o[2 * NB][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int cseq = -1, cunit = -1, cstep0 = 0;
    int stage = 0;
    uint32_t phase = 0;

    // The current unit's state leaves the registers: as its result when the
    // warp has seen all of it, else as a piece to be joined.
    auto leave = [&](bool to_end, bool last) {
#pragma unroll
      for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
        l[h] += __shfl_xor_sync(~0u, l[h], 1);
        l[h] += __shfl_xor_sync(~0u, l[h], 2);
      }
      const bool whole = cstep0 == 0 && to_end;
      const int kvh = cunit / a.head_groups, h0 = (cunit % a.head_groups) * ROWS;
      float *state = nullptr;
      if (!whole) {
        // (a range that ends here has consumed its ring: the state goes there)
        state = last ? reinterpret_cast<float *>(ring) : a.first + ((size_t)blockIdx.x * kAttMaxWarps + warp) * floats;
        if (lane == 0)
          piece[warp][cstep0 == 0 ? 1 : 0] = make_int4(cseq, cunit, (cstep0 ? 1 : 0) | (to_end ? 0 : 2), last ? 2 : 1);
      }
#pragma unroll
      for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
        const int r = row + 8 * h, hd = kvh * a.group + h0 + r;
        const bool live = h0 + r < a.group;
        float mul = 1.f;
        uint8_t *out = nullptr;
        if (whole) {
          if (live) {
            const Ends e = finish(a, hd, m[h], l[h]);
            mul = e.mul;
            if (a.lse && quad == 0) a.lse[(long long)cseq * a.n_heads + hd] = e.lse;
            out = a.out + cseq * a.ldo + (long long)hd * dim * 2;
          }
        } else if (quad == 0) {
          state[r] = m[h];
          state[ROWS + r] = l[h];
        }
        float *sums = state + 2 * ROWS + r * dim;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (ANY && b >= nb) continue;
          float x[4];  // n-tiles 2b and 2b + 1, columns 2 quad and 2 quad + 1
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float(&c)[4] = o[2 * b + (i >> 1)];
            x[i] = (WIDE ? c[(i & 1) + 2 * h] : c[i & 1] + c[(i & 1) + 2]) * mul;
          }
          if (TYPE == LORA_KV_BF16) {  // dims 16 b + 2 quad, + 1, + 8, + 9
            const int d = 16 * b + 2 * quad;
            if (whole) {
              if (live) {
                *reinterpret_cast<uint32_t *>(out + d * 2) = pack_bf16x2(x[0], x[1]);
                *reinterpret_cast<uint32_t *>(out + d * 2 + 16) = pack_bf16x2(x[2], x[3]);
              }
            } else {
              *reinterpret_cast<float2 *>(sums + d) = make_float2(x[0], x[1]);
              *reinterpret_cast<float2 *>(sums + d + 8) = make_float2(x[2], x[3]);
            }
          } else {  // n-tile 2b: even dims, 2b + 1: odd dims; 16 b + 4 quad ..
            const int d = 16 * b + 4 * quad;
            if (whole) {
              if (live) *reinterpret_cast<uint2 *>(out + d * 2) = make_uint2(pack_bf16x2(x[0], x[2]), pack_bf16x2(x[1], x[3]));
            } else {
              *reinterpret_cast<float4 *>(sums + d) = make_float4(x[0], x[2], x[1], x[3]);
            }
          }
        }
      }
    };

    for (long long i = w0; i < w1; ++i) {
      const int seq = __shfl_sync(~0u, d_seq, stage), unit = __shfl_sync(~0u, d_unit, stage);
      const int step = __shfl_sync(~0u, d_step, stage), len = __shfl_sync(~0u, d_len, stage);
      const int bad = __shfl_sync(~0u, d_bad, stage);
      if (seq != cseq || unit != cunit) {
        if (cseq >= 0) leave(true, false);
        cseq = seq;
        cunit = unit;
        cstep0 = step;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int n = 0; n < 2 * NB; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        // q as the products' A operand: rows = heads, columns = dims in the order of the K operand
        const int kvh = unit / a.head_groups, h0 = (unit % a.head_groups) * ROWS;
#pragma unroll
        for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
          const bool live = h0 + row + 8 * h < a.group;
          const uint8_t *q = a.q + seq * a.ldq + (long long)(kvh * a.group + h0 + row + 8 * h) * dim * 2;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            uint32_t lo = 0, hi = 0;
            if (live && (!ANY || b < nb)) {
              if (TYPE == LORA_KV_BF16) {  // dims 2 quad, + 1 and + 8, + 9
                lo = __ldg(reinterpret_cast<const uint32_t *>(q + b * 32 + quad * 4));
                hi = __ldg(reinterpret_cast<const uint32_t *>(q + b * 32 + quad * 4 + 16));
              } else {  // dims 4 quad, + 2 (the even bytes) and + 1, + 3 (the odd ones)
                const uint2 u = __ldg(reinterpret_cast<const uint2 *>(q + b * 32 + quad * 8));
                lo = __byte_perm(u.x, u.y, 0x5410);
                hi = __byte_perm(u.x, u.y, 0x7632);
              }
            }
            qa[b][WIDE ? h : 0] = lo;
            qa[b][WIDE ? 2 + h : 1] = hi;
          }
        }
      }
      if (!mbar_wait_bounded(&full[warp][stage], phase, kv.status)) {
        dead = true;
        break;
      }
      const uint32_t st32 = ring32 + stage * stage_bytes;
      uint8_t *st = ring + stage * stage_bytes;
      // tokens of the step that count: [lo, hi) of its 16 TT, without those on bad pages
      const int pos0 = (first_token(len, a.window) / kTileTokens + step * TT) * kTileTokens;
      const int lo = first_token(len, a.window) - pos0, hi = len - pos0;
      const bool partial = lo > 0 || hi < kTileTokens * TT || bad;
      if (TYPE == LORA_KV_BF16 && partial) {
        // weight 0 times what lies there must be 0: clear V's rows outside
        for (int t = 0; t < kTileTokens * TT; ++t) {
          if (t >= lo && t < hi && !(bad >> (t / kTileTokens) & 1)) continue;
          uint8_t *v = st + (t / kTileTokens) * tile_bytes + (kTileTokens + t % kTileTokens) * row_bytes;
          for (int c = lane; c < chunks; c += 32) *reinterpret_cast<uint4 *>(v + c * 16) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }

      // ---- scores: [heads] x [16 TT tokens]
      float c[2 * TT][4];
#pragma unroll
      for (int n = 0; n < 2 * TT; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint32_t k32 = st32 + t * tile_bytes + k_row;
        if (TYPE == LORA_KV_BF16) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            if (ANY && b >= nb) continue;
            uint32_t k[4];
            ldsm4(k, k32 + (((2 * b + k_c) ^ sw) << 4));
            if (WIDE) {
              mma16816(c[2 * t], qa[b][0], qa[b][1], qa[b][2 % (WIDE ? 4 : 2)], qa[b][3 % (WIDE ? 4 : 2)], k[0], k[1]);
              mma16816(c[2 * t + 1], qa[b][0], qa[b][1], qa[b][2 % (WIDE ? 4 : 2)], qa[b][3 % (WIDE ? 4 : 2)], k[2], k[3]);
            } else {
              mma16816(c[2 * t], qa[b][0], qa[b][0], qa[b][1], qa[b][1], k[0], k[1]);
              mma16816(c[2 * t + 1], qa[b][0], qa[b][0], qa[b][1], qa[b][1], k[2], k[3]);
            }
          }
        } else {
#pragma unroll
          for (int p = 0; p < (NB + 1) / 2; ++p) {
            if (ANY && 2 * p >= nb) continue;
            uint32_t w[4];
            ldsm4(w, k32 + (((2 * p + k_c) ^ sw) << 4));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int b = 2 * p + x;
              if (b >= NB || (ANY && b >= nb)) continue;
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t even, odd;
                codes_to_bf16<TYPE>(w[2 * x + y], even, odd);
                if (WIDE)
                  mma16816(c[2 * t + y], qa[b][0], qa[b][1], qa[b][2 % (WIDE ? 4 : 2)], qa[b][3 % (WIDE ? 4 : 2)], even, odd);
                else
                  mma16816(c[2 * t + y], qa[b][0], qa[b][0], qa[b][1], qa[b][1], even, odd);
              }
            }
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
          const uint8_t *sc = st + t * tile_bytes + 2 * kTileTokens * row_bytes;
          ks = *reinterpret_cast<const float2 *>(sc + tok * 4);
          ks.x *= a.scale2;
          ks.y *= a.scale2;
          const float2 u = *reinterpret_cast<const float2 *>(sc + (kTileTokens + tok) * 4);
          vs[n][0] = u.x;
          vs[n][1] = u.y;
        }
        c[n][0] *= ks.x;
        c[n][1] *= ks.y;
        if (WIDE) {
          c[n][2] *= ks.x;
          c[n][3] *= ks.y;
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
      float mx[2], base_m[2];
      bool moved = false;
#pragma unroll
      for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
        mx[h] = m[h];
#pragma unroll
        for (int n = 0; n < 2 * TT; ++n) mx[h] = fmaxf(mx[h], fmaxf(c[n][2 * h], c[n][2 * h + 1]));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(~0u, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(~0u, mx[h], 2));
        base_m[h] = mx[h] == -INFINITY ? 0.f : mx[h];
        moved |= mx[h] > m[h];
      }
      if (__any_sync(~0u, moved)) {
#pragma unroll
        for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
          const float alpha = exp2_fast(m[h] - base_m[h]);
          l[h] *= alpha;
          m[h] = mx[h];
#pragma unroll
          for (int n = 0; n < 2 * NB; ++n) {
            if (ANY && n >= 2 * nb) continue;
            if (WIDE) {
              o[n][2 * h] *= alpha;
              o[n][2 * h + 1] *= alpha;
            } else {
              o[n][0] *= alpha;
              o[n][1] *= alpha;
              o[n][2] *= alpha;
              o[n][3] *= alpha;
            }
          }
        }
      }
      uint32_t ph[2 * TT][WIDE ? 2 : 1], pl[2 * TT][WIDE ? 2 : 1];  // weights, and what their rounding left
#pragma unroll
      for (int n = 0; n < 2 * TT; ++n)
#pragma unroll
        for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
          float p0 = exp2_fast(c[n][2 * h] - base_m[h]), p1 = exp2_fast(c[n][2 * h + 1] - base_m[h]);
          l[h] += p0 + p1;
          if (TYPE != LORA_KV_BF16) {
            p0 *= vs[n][0];
            p1 *= vs[n][1];
          }
          ph[n][h] = pack_bf16x2(p0, p1);
          pl[n][h] = pack_bf16x2(p0 - bf16_lo(ph[n][h]), p1 - bf16_hi(ph[n][h]));
        }

      // ---- weighted values
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint32_t v32 = st32 + t * tile_bytes + kTileTokens * row_bytes + v_row;
        auto add = [&](float(&acc)[4], uint32_t b0, uint32_t b1) {
          if (WIDE) {
            mma16816(acc, ph[2 * t][0], ph[2 * t][WIDE ? 1 : 0], ph[2 * t + 1][0], ph[2 * t + 1][WIDE ? 1 : 0], b0, b1);
            mma16816(acc, pl[2 * t][0], pl[2 * t][WIDE ? 1 : 0], pl[2 * t + 1][0], pl[2 * t + 1][WIDE ? 1 : 0], b0, b1);
          } else {
            mma16816(acc, ph[2 * t][0], pl[2 * t][0], ph[2 * t + 1][0], pl[2 * t + 1][0], b0, b1);
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
              codes_to_bf16<TYPE>(w[2 * x], e0, o0);
              codes_to_bf16<TYPE>(w[2 * x + 1], e1, o1);
              add(o[2 * b], e0, e1);
              add(o[2 * b + 1], o0, o1);
            }
          }
        }
      }
      __syncwarp();  // (all lanes have read the stage)
      fetch(stage);
      if (++stage == a.n_stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!dead) {
      // (the fetching side is just past the range: at a unit's first step where the range ends with one)
      leave(fstep == 0, true);
    } else {
      // copies in flight must land before the block ends (again a bounded wait)
      for (int i = 0; i < a.n_stages; ++i) (void)mbar_wait_bounded(&full[warp][i], phase ^ (i < stage), kv.status);
      if (lane == 0) dead_block = 1;
    }
  }
  __syncthreads();

  // ---- join what the warps' borders cut
  const bool broken = dead_block != 0;
  // (pieces of one unit follow one another; entry = 2 * warp + which)
  if (tid == 0) {
    int n = 0, ch = -1, ps = -1, pu = -1;
    for (int w = 0; w < n_warps; ++w)
      for (int k = 0; k < 2; ++k) {
        const int4 p = piece[w][k];
        if (p.x < 0) continue;
        if (p.x != ps || p.y != pu) ++ch;
        ps = p.x;
        pu = p.y;
        list[n] = 2 * w + k;
        chain_of[n++] = ch;
      }
    n_pieces = n;
    n_chains = ch + 1;
    int4 cut = make_int4(-1, 0, 0, 0);
    if (n && !broken) {
      const int4 p = piece[list[n - 1] >> 1][list[n - 1] & 1];
      int f = n - 1;
      while (f > 0 && chain_of[f - 1] == ch) --f;
      const int4 q = piece[list[f] >> 1][list[f] & 1];
      if ((p.z & 2) && !(q.z & 1))  // goes on past the block, and starts in it; its last step's block:
        cut = make_int4(p.x, p.y, (int)((tail_end * blocks - 1) / steps_all), 0);
    }
    a.cut[blockIdx.x] = cut;
  }
  if (broken && tid < 2 * ROWS)  // (no result for what this block was to add to)
    a.part[((size_t)blockIdx.x * 2 + tid / ROWS) * floats + ROWS + tid % ROWS] = -1.f;
  __syncthreads();
  for (int task = warp; task < n_chains * ROWS; task += n_warps) {
    const int ch = task / ROWS, r = task % ROWS;
    int f = 0;
    while (chain_of[f] != ch) ++f;
    int e = f;
    while (e < n_pieces && chain_of[e] == ch) ++e;
    auto state_of = [&](int i) -> const float * {
      const int w = list[i] >> 1;
      return piece[w][list[i] & 1].w == 2 ? reinterpret_cast<const float *>(smem + (size_t)w * a.n_stages * stage_bytes)
                                          : a.first + ((size_t)blockIdx.x * kAttMaxWarps + w) * floats;
    };
    const int4 p0 = piece[list[f] >> 1][list[f] & 1], p1 = piece[list[e - 1] >> 1][list[e - 1] & 1];
    const int h0 = (p0.y % a.head_groups) * ROWS;
    if (h0 + r >= a.group) continue;
    float mm = -INFINITY;
    for (int i = f; i < e; ++i) mm = fmaxf(mm, state_of(i)[r]);
    const float bm = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f;
    float4 x[2] = {};  // dims 4 lane .., 128 + 4 lane ..
    for (int i = f; i < e; ++i) {
      const float *st = state_of(i);
      const float w = exp2_fast(st[r] - bm);
      ll += w * st[ROWS + r];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int d = 128 * k + 4 * lane;
        if (d >= dim) continue;
        const float4 y = *reinterpret_cast<const float4 *>(st + 2 * ROWS + r * dim + d);
        x[k].x = fmaf(w, y.x, x[k].x);
        x[k].y = fmaf(w, y.y, x[k].y);
        x[k].z = fmaf(w, y.z, x[k].z);
        x[k].w = fmaf(w, y.w, x[k].w);
      }
    }
    if (!(p0.z & 1) && !(p1.z & 2)) {  // all of the unit
      if (broken) continue;
      const int hd = (p0.y / a.head_groups) * a.group + h0 + r;
      const Ends fin = finish(a, hd, mm, ll);
      if (a.lse && lane == 0) a.lse[(long long)p0.x * a.n_heads + hd] = fin.lse;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int d = 128 * k + 4 * lane;
        if (d >= dim) continue;
        *reinterpret_cast<uint2 *>(a.out + p0.x * a.ldo + ((long long)hd * dim + d) * 2) =
            make_uint2(pack_bf16x2(x[k].x * fin.mul, x[k].y * fin.mul), pack_bf16x2(x[k].z * fin.mul, x[k].w * fin.mul));
      }
    } else {
      float *st = a.part + ((size_t)blockIdx.x * 2 + (p0.z & 1 ? 0 : 1)) * floats;
      if (lane == 0) {
        st[r] = mm;
        st[ROWS + r] = broken ? -1.f : ll;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int d = 128 * k + 4 * lane;
        if (d < dim) *reinterpret_cast<float4 *>(st + 2 * ROWS + r * dim + d) = x[k];
      }
    }
  }

  // ---- sequences without a token: zeros, or untouched (length -1, and lengths in error)
  for (int i0 = blockIdx.x + warp * 32 * gridDim.x; i0 < s.n; i0 += gridDim.x * blockDim.x) {
    const int i = i0 + lane * gridDim.x;
    int len = 1;
    if (i < s.n && i >= 0) {
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
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(AttendArgs a, int rows, int dim) {
  __shared__ float sums[kJoinThreads * 4];
  __shared__ float tops[16], lens[kJoinThreads];
  __shared__ int broken;
  griddep_wait();
  griddep_launch_dependents();
  const int4 cut = a.cut[blockIdx.x];
  if (cut.x < 0) return;
  const int floats = state_floats(rows, dim), n = cut.z - blockIdx.x + 1;
  auto state = [&](int i) { return a.part + ((size_t)(blockIdx.x + i) * 2 + (i ? 0 : 1)) * floats; };
  const int h0 = (cut.y % a.head_groups) * rows, live = min(rows, a.group - h0);
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
        const float4 y = *reinterpret_cast<const float4 *>(st + 2 * rows + r * dim + d);
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

template <int TYPE, int DIM, int TT>
Variant variant() {
  return {{attend_kernel<TYPE, DIM, TT, false>, attend_kernel<TYPE, DIM, TT, true>}, TT};
}

Variant variant_of(int type, int dim) {
  if (type == LORA_KV_BF16)
    return dim == 128 ? variant<LORA_KV_BF16, 128, 1>() : dim == 64 ? variant<LORA_KV_BF16, 64, 2>() : variant<LORA_KV_BF16, 256, 1>();
  if (type == LORA_KV_E4M3)
    return dim == 128 ? variant<LORA_KV_E4M3, 128, 2>() : dim == 64 ? variant<LORA_KV_E4M3, 64, 4>() : variant<LORA_KV_E4M3, 256, 1>();
  return dim == 128 ? variant<LORA_KV_INT8, 128, 2>() : dim == 64 ? variant<LORA_KV_INT8, 64, 4>() : variant<LORA_KV_INT8, 256, 1>();
}

constexpr int kAttStatic = 4096;  // at least what the kernel's static shared memory takes

// Warps and stages: at least 3 stages a warp, 8 warps where that fits.
void geometry(int stage_bytes, int *warps, int *stages) {
  const int room = kAttSmem - kAttStatic;
  *warps = room / (3 * stage_bytes);
  *warps = *warps > kAttMaxWarps ? kAttMaxWarps : *warps;
  *stages = room / (*warps * stage_bytes);
  *stages = *stages > kAttMaxStages ? kAttMaxStages : *stages;
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
  const int rows = group_of(kv, n_heads) > 8 ? 16 : 8;
  const size_t state = size_t(state_floats(rows, kv->dim)) * 4;
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
  const int rows = wide ? 16 : 8;
  a.head_groups = (a.group + rows - 1) / rows;
  a.units = kv->heads * a.head_groups;
  a.scale2 = c.scale * 1.44269504f;
  a.window = c.window;
  const int stage_bytes = v.tt * kv_tile_bytes(kv->type, kv->dim);
  int warps;
  geometry(stage_bytes, &warps, &a.n_stages);
  uint8_t *ws = static_cast<uint8_t *>(c.ws);
  const size_t floats = state_floats(rows, kv->dim);
  a.cut = reinterpret_cast<int4 *>(ws);
  a.part = reinterpret_cast<float *>(ws + align256(size_t(kv->n_sm) * sizeof(int4)));
  a.first = a.part + size_t(kv->n_sm) * 2 * floats;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kv->n_sm);
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = size_t(warps) * a.n_stages * stage_bytes;
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
  rc = cuda_status(cudaLaunchKernelEx(&cfg, attend_join_kernel, a, rows, kv->dim));
  if (rc == LORA_OK) g_launches.fetch_add(1);
  return rc;
}

}  // namespace lora
