// Attention over the 4-bit cache, few query rows at a time (decode, short
// prompts, fp32).
//
// A unit is one KV head of one sequence (dense: every token up to the query's
// position) or of one 64-query block (routed: the group list of hga_attend).
// Its query rows are (position, query head of the KV head) pairs, taken 8 * NT
// at a time as the columns of the products
//   S^T[token][row] = K[token][dim] Q^T[dim][row],  O^T[dim][row] = V^T[dim][token] P^T[token][row]
// with mma.sync m16n8k16 on fp16: tokens (then dims) fill the 16 wide side, so
// the 8 query heads of a group fill the other one and no half is padding.
// tcgen05 would pad 8 rows to 64 and want K and V expanded into shared
// memory first; here the codes go from the record straight into the operands'
// registers, 32 dims of a token per thread for K, 16 dims of 4 tokens for V
// (two tokens' nibbles are merged so that one conversion yields a token pair).
// Codes times scales are exact in fp16.  q enters as fp16 relative to a power
// of two of its row (bf16: exact up to 2^-25 of the row's maximum; fp32: as a
// sum of two fp16 values, like P, 22 bits).  Sums, maxima and O are fp32.
//
// Bound: no unit is full (issue slots 57 %, ALU 52 %, HBM 49 %): a warp's step is
// one chain of loads, conversions, products and softmax, and the registers allow
// 12 warps an SM.  8 sequences of 32K to 64K tokens, 32 heads on 4, d 128, with
// the append and the join: 66 us for 237 MB.  Each warp runs
// alone: it fetches 64 tokens (8 records) at a time into its own ring by bulk copies and
// never waits for another warp until the end, where the CTA's warps join their
// (max, sum, O), and a second kernel joins the splits of a long context, in a
// fixed order.
#pragma once
#include "attend.cuh"
#include "q4.cuh"
#include "tc.cuh"

namespace hga {

constexpr int kQ4Warps = 4;
constexpr int kQ4StepRecs = 8;            // records of 8 tokens a warp takes at a time
constexpr int kQ4StepTok = 8 * kQ4StepRecs;
// Weights are held as 2^11 times exp(score - m), m a maximum that is only moved
// when a score passes it by more than 2^4: at most 2^15 in fp16, with 11 bits
// down to 2^-25 of the largest one (fp16's subnormals start at 2^-14).
constexpr float kQ4PShift = 11.f, kQ4Grow = 4.f;

struct Q4AttendArgs {
  Q4Cache c;
  Q4BatchArgs b;
  AttendArgs a;            // routed: lists, blocks, sink, local, scale_log2 ... (dense: q, o, lse,
                           // Hq, Hkv, G, scale_log2)
  int max_q;               // dense: most query positions of a sequence
  int row;                 // routed: the sequence's table row
  int z0;                  // routed: the first block with rows to compute
  int n_split;             // CTAs a unit's tokens are split over
  int slots;               // dense, few rows: CTAs per KV head and tile that all the sequences'
                           // tokens are dealt out to (see q4_deal), 0 = one per sequence
  int n_tiles;             // row tiles a unit can have
  float shift;             // log2 of the factor that weights and their sums carry
  float* part_o;           // [unit][split][row][D] (n_split > 1) or [KV head][slot][tile][row][D]
  float2* part_ml;         // [unit][split][row]  max (log2 units), sum
};

template <int D, int NT, bool ROUTED>
struct Q4Layout {
  static constexpr int kStages = 2;
  static constexpr int kRec = q4_record_bytes(D);
  static constexpr int kStage = kQ4StepRecs * kRec;
  static constexpr int kRingOff = 0;
  static constexpr int kRing = kQ4Warps * kStages * kStage;
  static constexpr int kJoin = kQ4Warps * 8 * NT * (D + 2) * 4;     // reuses the ring
  static constexpr int kBarOff = kRing > kJoin ? kRing : kJoin;
  static constexpr int kEntOff = kBarOff + kQ4Warps * kStages * 8;   // [warp][stage][8] entries
  static constexpr size_t kSmem = kEntOff + kQ4Warps * kStages * 32;
};

__device__ __forceinline__ void q4_mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The 8x8 fp16 tile held one row per quad, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::
          "r"(tc::smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(tc::smem_addr(bar))
      : "memory");
}

// fp16 pair (hi) of two floats, and of what it leaves (lo).
__device__ __forceinline__ uint32_t split_half2(float x, float y, uint32_t* lo) {
  const uint32_t hi = tc::pack_half2(x, y);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  *lo = tc::pack_half2(x - f.x, y - f.y);
  return hi;
}

// A row's maximum M (log2 units) and sum of weights S.  A row that attends
// nothing has S = 0; a query that is not finite makes S NaN, and with it the
// output and lse; a score that fp32 does not hold makes M infinite.
__device__ __forceinline__ bool q4_nonfinite(float M, float S) {
  return S != 0.f && !(fabsf(M) + S <= 3.0e38f);
}
__device__ __forceinline__ float q4_inverse(float S) { return S == 0.f ? 0.f : 1.f / S; }
// shift: log2 of the factor that weights and their sums carry.
__device__ __forceinline__ float q4_lse(float M, float S, float shift) {
  return S == 0.f ? -INFINITY : (M + (log2f(S) - shift)) * 0.6931471805599453f;
}

// A unit's position in the batch, from the block index.
struct Q4Unit {
  int row;                 // table row, < 0: nothing to attend (outputs 0 and -inf)
  int64_t tok0;            // first query row of q / o of the unit's sequence or block
  int n;                   // query positions
  int pos0;                // position of the first one
  int ctx;                 // tokens the sequence has
};

__device__ __forceinline__ bool q4_unit(const Q4AttendArgs& g, bool routed, int z, Q4Unit* u) {
  if (routed) {
    const int64_t b0 = g.a.q_start + (int64_t)z * g.a.qblock;
    const int64_t T = g.a.q_start + g.a.n_q;
    const int skip = (int)max((int64_t)0, g.a.pos_lo - b0);   // rows before pos_lo are left
    u->row = g.row;
    u->n = (int)min((int64_t)g.a.qblock, T - b0) - skip;
    u->tok0 = (int64_t)z * g.a.qblock + skip;
    u->pos0 = (int)b0 + skip;
    u->ctx = (int)T;
    return u->n > 0;
  }
  const int r = g.b.rows[z];
  u->tok0 = g.b.off ? g.b.off[z] : z;
  u->n = g.b.off ? g.b.off[z + 1] - (int)u->tok0 : 1;
  if (u->n <= 0 || u->n > g.max_q || u->tok0 < 0 || u->tok0 + u->n > g.a.n_q) {
    if (u->n != 0) report(HGA_ERR_DEVICE_CHECK);
    return false;
  }
  u->row = r;
  u->ctx = 0;
  u->pos0 = 0;
  if (r >= g.c.n_rows) {
    report(HGA_ERR_DEVICE_CHECK);
    u->row = -1;
  }
  if (u->row >= 0) {
    u->ctx = g.c.len[r];
    u->pos0 = u->ctx - u->n;
    if (u->pos0 < 0 || u->ctx > (int64_t)g.c.row_pages * g.c.page_tokens) {
      report(HGA_ERR_DEVICE_CHECK);       // fewer tokens than queries
      u->row = -1;
    }
  }
  return true;
}

// The records that a unit attends, in order: dense, those of its tokens; routed,
// the sink, routed, local-window and diagonal groups of hga_attend.
struct Q4List {
  int n;                   // entries
  int n_whole;             // entries that every row attends whole
  int n_s, n_r, loc0, n_l, d0;
  int lo, hi;              // routed groups lie in [lo, hi)
  const int32_t* routed;
};

// dense: first_pos and last_pos are the positions of the first and last row.
template <bool ROUTED>
__device__ __forceinline__ Q4List q4_list(const Q4AttendArgs& g, const Q4Unit& u, int z, int h,
                                          int first_pos, int last_pos) {
  Q4List x{};
  if constexpr (ROUTED) {
    const int64_t b0 = g.a.q_start + (int64_t)z * g.a.qblock;
    const int64_t sink_end = min((int64_t)g.a.sink, b0);
    const int64_t loc_lo = max(sink_end, b0 - g.a.local);
    x.n_s = (int)(sink_end / 8);
    x.n_r = g.a.group_cnt[(int64_t)h * g.a.n_blocks + z];
    if (x.n_r < 0 || x.n_r > g.a.cap_g) {
      report(HGA_ERR_DEVICE_CHECK);
      x.n_r = 0;
    }
    x.loc0 = (int)(loc_lo / 8);
    x.n_l = (int)((b0 - loc_lo) / 8);
    x.d0 = (int)(b0 / 8);
    x.lo = g.a.sink / 8;
    x.hi = (int)((b0 - g.a.local) / 8);
    x.routed = g.a.group_idx + ((int64_t)h * g.a.n_blocks + z) * g.a.cap_g;
    x.n_whole = x.n_s + x.n_r + x.n_l;
    x.n = x.n_whole + (last_pos + 1 - (int)b0 + 7) / 8;
  } else if (u.row >= 0) {
    x.n = (last_pos >> 3) + 1;
    x.n_whole = (first_pos + 1) >> 3;
  }
  return x;
}

// Entry i (a record of the sequence), -1 where there is none: past the end, or
// a routed group that is not legal (reported).
template <bool ROUTED>
__device__ __forceinline__ int q4_entry(const Q4List& x, int i) {
  if (i < 0 || i >= x.n) return -1;
  if constexpr (!ROUTED) return i;
  if (i < x.n_s) return i;
  int r = i - x.n_s;
  if (r < x.n_r) {
    const int e = x.routed[r], before = r > 0 ? x.routed[r - 1] : -1;
    if (e >= x.lo && e < x.hi && e > before) return e;
    report(HGA_ERR_DEVICE_CHECK);
    return -1;
  }
  r -= x.n_r;
  return r < x.n_l ? x.loc0 + r : x.d0 + r - x.n_l;
}

// Where a record lies, in two halves so that nothing waits for the page table
// until a step later: its page (as the table says, -1 past the row) and its index
// in the page; then the byte offset from the plane's first page, -1 (reported)
// where the table names none.
__device__ __forceinline__ int q4_page_of(const Q4Cache& c, const int32_t* pages, int ent, int* in) {
  // ent / page_recs by the reciprocal, off by at most one
  int col = (int)__umulhi((uint32_t)ent, c.page_recs_inv);
  *in = ent - col * c.page_recs;
  if (*in < 0) --col, *in += c.page_recs;
  else if (*in >= c.page_recs) ++col, *in -= c.page_recs;
  return col < c.row_pages ? pages[col] : -1;
}
__device__ __forceinline__ int64_t q4_offset(const Q4Cache& c, int h, int page, int in,
                                             int rec_bytes) {
  if (page < 0 || page >= c.n_pages) {
    report(HGA_ERR_DEVICE_CHECK);
    return -1;
  }
  return page * c.page_bytes + ((int64_t)h * c.page_recs + in) * rec_bytes;
}

// Fetches up to 8 records (lane e < 8 holds record e's offset, -1 for none) to
// dst + e * rec.  Records that follow one another in memory come in one copy:
// a copy's cost is in its issue (one of 576 or 1152 bytes per record kept the
// expanding warps of q4_attend_tc.cuh waiting for 60% of the time).  Arms bar:
// lane 0's arrive comes after every lane's stores so far (other warps read the
// load's entries once bar completes, which is at once where no record is there).
__device__ __forceinline__ void q4_fetch8(char* dst, const char* base, int64_t at, int rec,
                                          uint64_t* bar, int lane) {
  const int64_t before = __shfl_up_sync(0xffffffffu, at, 1);
  const unsigned live = __ballot_sync(0xffffffffu, at >= 0);
  const bool first = at >= 0 && (lane == 0 || before < 0 || at != before + rec);
  const unsigned stops = __ballot_sync(0xffffffffu, first) | ~live;
  __syncwarp();
  if (lane == 0) tc::mbar_arrive_expect_tx(bar, __popc(live) * rec);
  __syncwarp();
  if (first) {
    const unsigned after = stops & (0xfffffffeu << lane);
    bulk_load(dst + lane * rec, base + at, (__ffs(after) - 1 - lane) * rec, bar);
  }
}

// The batch's tokens dealt out to `slots` CTAs (more than sequences): every
// sequence gets as many as its length needs at `per` steps each, at least one,
// with a `per` that always suffices: sum ceil(steps / per) <= n_seq + total / per.
// It is not the least one: with lengths between half and all of the longest it
// is up to 1.1 times that for 8 sequences on 111 CTAs, 1.6 times for 32 on 55.  Only
// the device knows the lengths, and a split into as many parts for every
// sequence leaves the longest ones' CTAs running last.
__device__ __forceinline__ int q4_seq_steps(const Q4AttendArgs& g, int z) {
  const int r = g.b.rows[z];
  if (r < 0 || r >= g.c.n_rows) return 0;
  const int ctx = g.c.len[r];
  return ctx <= 0 || ctx > (int64_t)g.c.row_pages * g.c.page_tokens ? 0
                                                                        : (ctx + kQ4StepTok - 1) / kQ4StepTok;
}
__device__ __forceinline__ int q4_deal(const Q4AttendArgs& g, int lane) {
  int64_t total = 0;
  for (int z = lane; z < g.b.n_seq; z += 32) total += q4_seq_steps(g, z);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) total += __shfl_xor_sync(0xffffffffu, total, x);
  const int64_t spare = g.slots - g.b.n_seq;
  return (int)max((int64_t)kQ4Warps, (total + spare - 1) / spare);
}
// Which sequence and part of it a slot has (find = -1), or the first slot of
// sequence `find`.  False: the slot has none.
__device__ __forceinline__ bool q4_dealt(const Q4AttendArgs& g, int per, int lane, int find, int* slot,
                                         int* z) {
  int base = 0;
  for (int z0 = 0; z0 < g.b.n_seq; z0 += 32) {
    const int n = z0 + lane < g.b.n_seq ? max(1, (q4_seq_steps(g, z0 + lane) + per - 1) / per) : 0;
    int incl = n;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, x);
      if (lane >= x) incl += y;
    }
    const int all = __shfl_sync(0xffffffffu, incl, 31);
    if (find >= 0 ? find < z0 + 32 : *slot < base + all) {
      const unsigned past = __ballot_sync(0xffffffffu, *slot < base + incl);
      const int at = find >= 0 ? find - z0 : __ffs(past) - 1;
      const int first = base + __shfl_sync(0xffffffffu, incl - n, at);
      *z = z0 + at;
      *slot = find >= 0 ? first : *slot - first;
      return true;
    }
    base += all;
  }
  return false;
}

// Steps of one split.
__device__ __forceinline__ void q4_split_range(int steps, int n_split, int split, int* lo, int* hi) {
  const int per = (steps + n_split - 1) / n_split;
  *lo = min(steps, split * per);
  *hi = min(steps, *lo + per);
}

// CTAs of an SM: what the registers allow (the rings leave room for three).
// The loads, conversions and products of a step are one chain in a warp, so
// the more warps the better.
template <int NT, typename T>
constexpr int q4_ctas() { return NT == 1 && sizeof(T) == 2 ? 3 : 2; }

template <int D, int NT, typename T, bool ROUTED>
__global__ void __launch_bounds__(32 * kQ4Warps, (q4_ctas<NT, T>())) q4_attend_kernel(const Q4AttendArgs g) {
  using L = Q4Layout<D, NT, ROUTED>;
  constexpr int kQ4Stages = L::kStages;
  constexpr bool kSplitFp = sizeof(T) == 4;     // fp32: q and P as sums of two fp16 values
  constexpr int KS = D / 16;                    // k-steps of S, m-tiles of O
  constexpr int R = 8 * NT;
  constexpr int kMt = kQ4StepRecs / 2;          // 16-token tiles of a step
  extern __shared__ __align__(128) char smem[];
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gr = lane >> 2, t = lane & 3;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff) + warp * kQ4Stages;
  char* ring = smem + L::kRingOff + warp * kQ4Stages * L::kStage;
  int* ents = reinterpret_cast<int*>(smem + L::kEntOff) + warp * kQ4Stages * 8;

  if (tid == 0) s_abort = 0;
  if (lane == 0) {
    for (int s = 0; s < kQ4Stages; ++s) tc::mbar_init(&bars[s], 1);
    tc::fence_mbar_init();
  }
  __syncthreads();                              // every warp's waits read s_abort
  griddep_wait();
  const int h = blockIdx.y;
  const int n_x = !ROUTED && g.slots ? g.slots : g.n_split;
  const int tile = blockIdx.x / n_x;
  int split = blockIdx.x % n_x;
  int z = blockIdx.z + (ROUTED ? g.z0 : 0), per = 0;
  int64_t part = (((int64_t)blockIdx.z * gridDim.y + h) * g.n_tiles + tile) * n_x + split;
  if (!ROUTED && g.slots) {
    part = ((int64_t)h * n_x + split) * g.n_tiles + tile;
    per = q4_deal(g, lane);
    if (!q4_dealt(g, per, lane, -1, &split, &z)) return;
  }
  Q4Unit u;
  if (!q4_unit(g, ROUTED, z, &u)) return;
  const int nrows = u.n * g.a.G;
  const int row0 = tile * R;
  if (row0 >= nrows) return;
  const int last_pos = u.pos0 + min(nrows - 1, row0 + R - 1) / g.a.G;
  const int first_pos = u.pos0 + row0 / g.a.G;
  const Q4List list = q4_list<ROUTED>(g, u, z, h, first_pos, last_pos);
  const int n_ent = list.n;
  const int steps = (n_ent + kQ4StepRecs - 1) / kQ4StepRecs;
  int lo, hi;
  if (per) {
    lo = min(steps, split * per);
    hi = min(steps, lo + per);
  } else {
    q4_split_range(steps, g.n_split, split, &lo, &hi);
  }
  if (lo >= hi && split > 0) return;            // the join reads only splits with tokens
  const bool whole = per ? steps <= per : g.n_split == 1;   // nothing to join

  // ---- the warp's loads: lane l < 8 fetches record l of a step
  const int32_t* pages = g.c.table + (int64_t)max(u.row, 0) * g.c.row_pages;
  const int n_mine = hi > lo + warp ? (hi - lo - warp + kQ4Warps - 1) / kQ4Warps : 0;
  unsigned got[kQ4Stages];                      // records that were fetched, per stage
  int issued = 0;
  int ent = -1, page = -1, in = 0;              // this lane's record of the next fetch
  auto look = [&](int i) {
    ent = i < n_mine && lane < kQ4StepRecs
              ? q4_entry<ROUTED>(list, (lo + warp + i * kQ4Warps) * kQ4StepRecs + lane)
              : -1;
    if (ent >= 0) page = q4_page_of(g.c, pages, ent, &in);
  };
  // Fetches step i; its places were looked up during the step before.
  auto fetch = [&](int i, int s) -> unsigned {
    const int64_t at = ent >= 0 ? q4_offset(g.c, h, page, in, L::kRec) : -1;
    if (lane < kQ4StepRecs) ents[s * 8 + lane] = at >= 0 ? ent : -1;
    const unsigned m = __ballot_sync(0xffffffffu, at >= 0);
    ++issued;
    q4_fetch8(ring + s * L::kStage, g.c.base, at, L::kRec, &bars[s], lane);
    look(i + 1);
    return m;
  };
  look(0);
#pragma unroll
  for (int s = 0; s < kQ4Stages; ++s) got[s] = s < n_mine ? fetch(s, s) : 0;

  // ---- q: thread (gr, t) holds the dims D/4 t .. of row gr, relative to a power of two
  uint32_t qf[NT][KS][2], ql[kSplitFp ? NT : 1][kSplitFp ? KS : 1][2];
  float sc[NT][2];                              // scores' scale of rows 2t, 2t + 1 (log2 units)
  int pos[NT][2];                               // their positions
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = row0 + nt * 8 + gr;
    float f[D / 4];
    if (r < nrows) {
      const T* src = static_cast<const T*>(g.a.q) +
                     ((u.tok0 + r / g.a.G) * g.a.Hq + (int64_t)h * g.a.G + r % g.a.G) * D + t * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) q4_load16(src + 16 * i, f + 16 * i);
    } else {
#pragma unroll
      for (int i = 0; i < D / 4; ++i) f[i] = 0.f;
    }
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < D / 4; ++i) mx = fmaxf(mx, fabsf(f[i]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // 2^-e and 2^e with the row's maximum in [1, 2) after scaling (e in
    // [-126, 126]; a zero row takes 1; a row with an infinity becomes NaN, as
    // its softmax is)
    int ex = (int)((__float_as_uint(mx) >> 23) & 0xff);
    const bool inf = ex == 255;
    ex = mx == 0.f ? 127 : min(max(ex, 1), 253);
    const float down = __uint_as_float(inf ? 0x7fffffffu : (uint32_t)(254 - ex) << 23);
    const float up = __uint_as_float((uint32_t)ex << 23);
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float p = f[4 * j + 2 * x] * down, q = f[4 * j + 2 * x + 1] * down;
        if constexpr (kSplitFp) qf[nt][j][x] = split_half2(p, q, &ql[nt][j][x]);
        else qf[nt][j][x] = tc::pack_half2(p, q);
      }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      // the column 2t + x of the products is the row held by lanes 4 (2t + x) ..
      sc[nt][x] = __shfl_sync(0xffffffffu, up, 4 * (2 * t + x)) * g.a.scale_log2;
      pos[nt][x] = u.pos0 + min(nrows - 1, row0 + nt * 8 + 2 * t + x) / g.a.G;
    }
  }

  float o[KS][NT][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int i = 0; i < KS; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[i][nt][x] = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;

  // Token of S^T's row r (0..7) within its record: rows 2t and 2t + 1 are
  // tokens t and t + 4, so that the V loads of a quad touch four neighbouring
  // rows.
  const int tok_k = (gr >> 1) + 4 * (gr & 1);
  bool ok = true;
  for (int i = 0; ok && i < n_mine; ++i) {
    const int s = i % kQ4Stages;
    if (!(ok = tc::mbar_wait_warp(&bars[s], (i / kQ4Stages) & 1, &s_abort))) break;
    const char* st = ring + s * L::kStage;
    unsigned have = got[0];
#pragma unroll
    for (int x = 1; x < kQ4Stages; ++x) if (s == x) have = got[x];
    const int e0 = (lo + warp + i * kQ4Warps) * kQ4StepRecs;
    const bool edge = have != (1u << kQ4StepRecs) - 1 || e0 + kQ4StepRecs > list.n_whole;
    const int* ent_of = ents + s * 8;
    // ---- scores
    float sv[kMt][NT][4];
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) sv[mt][nt][x] = 0.f;
      const char* ra = st + (2 * mt) * L::kRec + tok_k * (D / 2) + t * (D / 8);
      const char* rb = ra + L::kRec;
      uint32_t wa[D / 32], wb[D / 32], sa[D / 64], sb[D / 64];
      const char* sp = st + (2 * mt) * L::kRec + 8 * D + tok_k * (D / 16) + t * (D / 64);
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(ra), y = *reinterpret_cast<const uint4*>(rb);
        wa[0] = x.x; wa[1] = x.y; wa[2] = x.z; wa[3] = x.w;
        wb[0] = y.x; wb[1] = y.y; wb[2] = y.z; wb[3] = y.w;
        const uint32_t p = *reinterpret_cast<const uint16_t*>(sp);
        const uint32_t q = *reinterpret_cast<const uint16_t*>(sp + L::kRec);
        sa[0] = (p & 0xff) * 0x00800080u; sa[1] = (p >> 8) * 0x00800080u;
        sb[0] = (q & 0xff) * 0x00800080u; sb[1] = (q >> 8) * 0x00800080u;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(ra), y = *reinterpret_cast<const uint2*>(rb);
        wa[0] = x.x; wa[1] = x.y;
        wb[0] = y.x; wb[1] = y.y;
        sa[0] = *reinterpret_cast<const uint8_t*>(sp) * 0x00800080u;
        sb[0] = *reinterpret_cast<const uint8_t*>(sp + L::kRec) * 0x00800080u;
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        uint32_t ha[4], hb[4];
        q4_unpack8(wa[w], ha);
        q4_unpack8(wb[w], hb);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          ha[x] = q4_mul2(ha[x], sa[w / 2]);
          hb[x] = q4_mul2(hb[x], sb[w / 2]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t af[4] = {ha[2 * x], hb[2 * x], ha[2 * x + 1], hb[2 * x + 1]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            q4_mma(sv[mt][nt], af, qf[nt][2 * w + x][0], qf[nt][2 * w + x][1]);
            if constexpr (kSplitFp)
              q4_mma(sv[mt][nt], af, ql[nt][2 * w + x][0], ql[nt][2 * w + x][1]);
          }
        }
      }
    }
    // ---- mask: tokens past the row's position and records that are not there
    if (edge) {
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int rec = 2 * mt + y;
          const int ent = ent_of[rec];
          const bool there = ent >= 0;
          const int tok = ent * 8 + tok_k;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (!there || tok > pos[nt][x]) sv[mt][nt][2 * y + x] = -INFINITY;
        }
    }
    // ---- softmax over the step's tokens.  m is a score, not yet scaled: the
    // difference to it is taken first, so that it stays <= 0 however large
    // scores are
    uint32_t ph[kMt][NT][2], pl[kSplitFp ? kMt : 1][NT][2];
    float top[NT][2];
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float mx = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt) mx = fmaxf(mx, fmaxf(sv[mt][nt][x], sv[mt][nt][2 + x]));
        top[nt][x] = mx;
        grow |= m[nt][x] == -INFINITY ? mx > -INFINITY : (mx - m[nt][x]) * sc[nt][x] > kQ4Grow;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float mx = top[nt][x];
#pragma unroll
          for (int q = 4; q < 32; q <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, q));
          const float mn = fmaxf(m[nt][x], mx);
          const float corr = mn == -INFINITY ? 1.f : tc::ex2((m[nt][x] - mn) * sc[nt][x]);
          m[nt][x] = mn;
          l[nt][x] *= corr;
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            o[j][nt][x] *= corr;
            o[j][nt][2 + x] *= corr;
          }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float use = m[nt][x] == -INFINITY ? 0.f : m[nt][x];
        float sum = 0.f;
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float& p = sv[mt][nt][2 * y + x];
            p = tc::ex2(fmaf(p - use, sc[nt][x], kQ4PShift));
            sum += p;
          }
        l[nt][x] += sum;
      }
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if constexpr (kSplitFp) {
            uint32_t lo2;
            ph[mt][nt][y] = transpose8(split_half2(sv[mt][nt][2 * y], sv[mt][nt][2 * y + 1], &lo2));
            pl[mt][nt][y] = transpose8(lo2);
          } else {
            ph[mt][nt][y] = transpose8(tc::pack_half2(sv[mt][nt][2 * y], sv[mt][nt][2 * y + 1]));
          }
        }
    }
    // ---- O^T += V^T P^T
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt) {
      // tokens k = 2t, 2t + 1 (record 2mt, tokens t and t + 4) and 2t + 8, 2t + 9
      uint32_t w[4][D / 64], sab, scd;
      const char* rec = st + (2 * mt) * L::kRec + 4 * D;
      const char* ssc = st + (2 * mt) * L::kRec + 8 * D + D / 2;
      uint32_t b4[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int tk = t + 4 * (y & 1);
        const char* at = rec + (y >> 1) * L::kRec + tk * (D / 2) + gr * (D / 16);
        if constexpr (D == 128) {
          const uint2 x = *reinterpret_cast<const uint2*>(at);
          w[y][0] = x.x; w[y][1] = x.y;
        } else {
          w[y][0] = *reinterpret_cast<const uint32_t*>(at);
        }
        b4[y] = *reinterpret_cast<const uint8_t*>(ssc + (y >> 1) * L::kRec + tk * (D / 16) +
                                                  (D == 128 ? gr : gr >> 1));
        if (edge) {
          // tokens that no row attends may hold anything: 0 * scale 0
          const int r = 2 * mt + (y >> 1);
          const int ent = ent_of[r];
          if (ent < 0 || ent * 8 + tk > last_pos) b4[y] = 0;
        }
      }
      sab = b4[0] << 7 | b4[1] << 23;
      scd = b4[2] << 7 | b4[3] << 23;
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        // byte j of lo: dim 2j of both tokens; of hi: dim 2j + 1
        const uint32_t k = 0x0f0f0f0fu;
        const uint32_t ab_lo = (w[0][x] & k) | ((w[1][x] << 4) & ~k);
        const uint32_t ab_hi = ((w[0][x] >> 4) & k) | (w[1][x] & ~k);
        const uint32_t cd_lo = (w[2][x] & k) | ((w[3][x] << 4) & ~k);
        const uint32_t cd_hi = ((w[2][x] >> 4) & k) | (w[3][x] & ~k);
        uint32_t f0[4], f1[4], f2[4], f3[4];
        q4_unpack8(ab_lo, f0);
        q4_unpack8(ab_hi, f1);
        q4_unpack8(cd_lo, f2);
        q4_unpack8(cd_hi, f3);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t af[4] = {q4_mul2(f0[j], sab), q4_mul2(f1[j], sab), q4_mul2(f2[j], scd),
                                  q4_mul2(f3[j], scd)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            q4_mma(o[4 * x + j][nt], af, ph[mt][nt][0], ph[mt][nt][1]);
            if constexpr (kSplitFp) q4_mma(o[4 * x + j][nt], af, pl[mt][nt][0], pl[mt][nt][1]);
          }
        }
      }
    }
    // ---- the stage is free: fetch the step after next
    __syncwarp();
    if (i + kQ4Stages < n_mine) {
      const unsigned f = fetch(i + kQ4Stages, s);
#pragma unroll
      for (int x = 0; x < kQ4Stages; ++x) if (s == x) got[x] = f;
    }
  }
  if (!ok) {
    // gave up: let the copies in flight land before the block's memory goes
    for (int s = 0; s < kQ4Stages && s < issued; ++s) {
      const uint64_t t0 = tc::globaltimer_ns();
      const int phase = (issued - 1 - s) / kQ4Stages;
      while (!tc::mbar_try_wait(&bars[s], phase & 1) &&
             tc::globaltimer_ns() - t0 < tc::kWaitLimitNs) {
      }
    }
  }
  // ---- join the warps: (max, sum, O) of each through shared memory
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int q = 4; q < 32; q <<= 1) l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], q);
  __syncthreads();                              // every warp is done with its ring
  float* jo = reinterpret_cast<float*>(smem);   // [warp][R][D]
  float2* jm = reinterpret_cast<float2*>(smem + kQ4Warps * R * D * 4);   // [warp][R]
  if (n_mine > 0) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = nt * 8 + 2 * t + x;
        if (gr == 0) {
          const float M = m[nt][x] * sc[nt][x];
          if (q4_nonfinite(M, l[nt][x])) report(HGA_ERR_DEVICE_CHECK);
          jm[warp * R + r] = make_float2(M, l[nt][x]);
        }
        float* dst = jo + (warp * R + r) * D + gr * (D / 8);
#pragma unroll
        for (int j = 0; j < KS; ++j)
          *reinterpret_cast<float2*>(dst + 2 * j) = make_float2(o[j][nt][x], o[j][nt][2 + x]);
      }
  }
  __syncthreads();
  const int n_w = min(kQ4Warps, hi - lo);       // warps that had a step
  for (int i = tid; i < R * (D / 4); i += 32 * kQ4Warps) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    if (row0 + r >= nrows) continue;
    float M = -INFINITY, S = 0.f;
    for (int w = 0; w < n_w; ++w) M = fmaxf(M, jm[w * R + r].x);
    const float use = M == -INFINITY ? 0.f : M;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < n_w; ++w) {
      const float2 ml = jm[w * R + r];
      const float f = tc::ex2(ml.x - use);
      const float4 v = *reinterpret_cast<const float4*>(jo + (w * R + r) * D + c);
      S += ml.y * f;
      acc.x += v.x * f; acc.y += v.y * f; acc.z += v.z * f; acc.w += v.w * f;
    }
    const int pr = row0 + r;
    if (!whole) {
      const int64_t at = part * R + r;
      *reinterpret_cast<float4*>(g.part_o + at * D + c) = acc;
      if (c == 0) g.part_ml[at] = make_float2(M, S);
      continue;
    }
    const float inv = q4_inverse(S);
    const int64_t orow = (u.tok0 + pr / g.a.G) * g.a.Hq + (int64_t)h * g.a.G + pr % g.a.G;
    T* dst = static_cast<T*>(g.a.o) + orow * D + c;
    dst[0] = Elt<T>::from_f32(acc.x * inv);
    dst[1] = Elt<T>::from_f32(acc.y * inv);
    dst[2] = Elt<T>::from_f32(acc.z * inv);
    dst[3] = Elt<T>::from_f32(acc.w * inv);
    if (c == 0 && g.a.lse) g.a.lse[orow] = q4_lse(M, S, kQ4PShift);
  }
  griddep_launch();
}

// Joins the splits of each unit's rows, in a fixed order.  R: rows of a tile,
// ENT: entries of a split's step.  Few rows (many splits each): a block of four
// warps joins one row, a warp every fourth split.  256 rows (few splits): 16
// rows a block, four for each warp.
template <int D, int R, int ENT, typename T, bool ROUTED>
__global__ void __launch_bounds__(128) q4_join_kernel(const Q4AttendArgs g) {
  constexpr int RB = R > 16 ? 16 : 1;
  constexpr int W = RB == 1 ? 4 : 1;            // warps of a row
  constexpr int V = D / 32;                     // values of a lane
  __shared__ float s_acc[4][D + 1];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tile = blockIdx.x / (R / RB), r_lo = blockIdx.x % (R / RB) * RB, h = blockIdx.y;
  Q4Unit u;
  const int z = blockIdx.z + (ROUTED ? g.z0 : 0);
  if (!q4_unit(g, ROUTED, z, &u)) return;
  const int nrows = u.n * g.a.G, row0 = tile * R;
  if (row0 + r_lo >= nrows) return;
  const int n_ent = q4_list<ROUTED>(g, u, z, h, u.pos0 + row0 / g.a.G,
                                    u.pos0 + min(nrows - 1, row0 + R - 1) / g.a.G).n;
  const int steps = (n_ent + ENT - 1) / ENT;
  int per = max(1, (steps + g.n_split - 1) / g.n_split);
  int64_t part0 = (((int64_t)blockIdx.z * gridDim.y + h) * g.n_tiles + tile) * g.n_split, stride = R;
  if (!ROUTED && g.slots) {
    int slot = 0, zz;
    per = q4_deal(g, lane);
    if (steps <= per) return;                          // already whole
    q4_dealt(g, per, lane, z, &slot, &zz);
    part0 = ((int64_t)h * g.slots + slot) * g.n_tiles + tile;
    stride = (int64_t)g.n_tiles * R;
  }
  const int n_s = max(1, (steps + per - 1) / per);     // splits that had tokens
  for (int r = r_lo + (W == 1 ? warp : 0); r < r_lo + RB && row0 + r < nrows; r += 4 / W) {
    const int64_t at0 = part0 * R + r;
    float M = -INFINITY;
    for (int s = lane; s < n_s; s += 32) M = fmaxf(M, g.part_ml[at0 + s * stride].x);
    M = warp_max(M);
    const float use = M == -INFINITY ? 0.f : M;
    float acc[V], S = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll 4
    for (int s = W == 1 ? 0 : warp; s < n_s; s += W) {
      const int64_t at = at0 + s * stride;
      const float2 ml = g.part_ml[at];
      const float f = tc::ex2(ml.x - use);
      S += ml.y * f;
      const float* src = g.part_o + at * D + lane * V;
      float v[V];
      if constexpr (V == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        v[0] = x.x; v[1] = x.y;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += v[i] * f;
    }
    if constexpr (W > 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) s_acc[warp][lane * V + i] = acc[i];
      if (lane == 0) s_acc[warp][D] = S;
      __syncthreads();
      if (warp > 0) return;
      S = 0.f;
      for (int w = 0; w < 4; ++w) S += s_acc[w][D];
#pragma unroll
      for (int i = 0; i < V; ++i)
        acc[i] = (s_acc[0][lane * V + i] + s_acc[1][lane * V + i]) +
                 (s_acc[2][lane * V + i] + s_acc[3][lane * V + i]);
    }
    const float inv = q4_inverse(S);
    const int pr = row0 + r;
    const int64_t orow = (u.tok0 + pr / g.a.G) * g.a.Hq + (int64_t)h * g.a.G + pr % g.a.G;
    T* dst = static_cast<T*>(g.a.o) + orow * D + lane * V;
#pragma unroll
    for (int i = 0; i < V; ++i) dst[i] = Elt<T>::from_f32(acc[i] * inv);
    if (lane == 0 && g.a.lse) g.a.lse[orow] = q4_lse(M, S, g.shift);
  }
  griddep_launch();
}

}  // namespace hga
