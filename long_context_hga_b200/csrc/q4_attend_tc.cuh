// Attention over the 4-bit cache with many query rows (prompts, routed blocks;
// bf16) on the sm_100a tensor cores: tcgen05.mma with TMEM accumulators.
//
// Units, query rows and entries are those of q4_attend.cuh.  A CTA takes 256
// rows of a unit as two 128-row tiles Q0/Q1 and walks its tokens 128 (16
// records) a step:
//   S_i = Q_i K^T,  O_i += P_i V       (fp16 operands, fp32 accumulators)
// K and V are expanded to fp16 on their way into shared memory, where a code
// times its scale is exact, so nothing is rounded there.  Q enters as fp16
// relative to a power of two of its row (see q4_attend.cuh).
//
// Warp roles (512 threads, registers split 80 : 176):
//   warp 0       TMEM owner and MMA issuer
//   warps 1-2    fetch records, 8 at a time by turns, into a ring by bulk copies
//   warps 4-7    expand: convert codes into the 128-byte swizzled operand
//                layout; tokens past the sequence and missing pages become zeros
//   warps 8-15   softmax of Q0 and Q1, one thread per row (of every 16
//                exponentials 4 are a polynomial on the FMA pipe)
// TMEM columns: S0 [0,128) S1 [128,256) (P over the first half of its S),
// O0 [256,256+D) O1 [384,384+D).
//
// A tile's chain is softmax, P V, next S; while one tile is in softmax the
// other's products run.  P V starts on the first 64 tokens while the others'
// weights are computed.  Bound: that chain (a step takes 4200 cycles, its
// products 2048).  3 sequences of up to 1K tokens on up to 8K, 32 heads on 8, d
// 128, with the append: 377 us, 0.49 of the bf16 rate; routed, 2K queries of a
// 64K context, 32 heads on 4: 61 us.
//
// Weights are held as 2^7 exp(score - m), m the running maximum, which is only
// moved when it grows by more than 2^8 (so that O is rarely rescaled): at most
// 2^15 in fp16, with 11 bits down to 2^-21 of the largest weight.
#pragma once
#include "attend_tc.cuh"
#include "q4_attend.cuh"

namespace hga {

constexpr int kQ4TcThreads = 512;
constexpr int kQ4TcLaunchRegs = 128, kQ4TcSoftmaxRegs = 176, kQ4TcOtherRegs = 80;
static_assert(256 * (kQ4TcSoftmaxRegs + kQ4TcOtherRegs) <= kQ4TcThreads * kQ4TcLaunchRegs,
              "register split");
constexpr int kQ4TcRows = 256;
constexpr int kQ4TcExpand = 128;           // threads that expand K and V
constexpr int kQ4TcSlots = 2;              // expanded K (and V) steps in shared memory
constexpr float kQ4TcShift = 7.f;

// A warp arrives once, after every lane's fence.
struct Q4TcBars {
  uint64_t q_full, k_full[kQ4TcSlots], k_empty[kQ4TcSlots], v_full[kQ4TcSlots],
      v_empty[kQ4TcSlots];
  uint64_t s_full[2], o_full[2], done;     // per Q tile
  uint64_t p_full[2][2];                   // [Q tile][half of the step's tokens]
  uint64_t raw_full[3], raw_empty[3];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Q4TcBars) <= 512, "barriers");

template <int D>
struct Q4TcLayout {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalfBytes = kTcRows * 128;
  static constexpr int kQBytes = 2 * kHalves * kHalfBytes;
  static constexpr int kGroupBytes = kHalves * 8 * 128;  // one record's K or V, expanded
  static constexpr int kSlotBytes = 16 * kGroupBytes;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + kQBytes;
  static constexpr int kVOff = kKOff + kQ4TcSlots * kSlotBytes;
  static constexpr int kBarOff = kVOff + kQ4TcSlots * kSlotBytes;
  static constexpr int kEntOff = kBarOff + 512;          // [8][8] entries, [8] flags
  static constexpr int kRawOff = kEntOff + 384;
  static constexpr int kRaw = 8 * q4_record_bytes(D);    // a stage: 8 records
  static constexpr int kStages = 3;
  static constexpr size_t kSmem = 1024 + (size_t)kRawOff + kStages * kRaw;
};
static_assert(Q4TcLayout<128>::kSmem <= 227 * 1024, "shared memory");

// 32 codes (16 bytes) with two scale bytes -> 64 bytes of a row of the operand
// layout, as four 16-byte chunks with the row's swizzle.  flip: the chunks are
// written in the order 2, 3, 0, 1 (the threads of the other 64 dims, whose rows
// lie in the same banks, write 0 .. 3).
__device__ __forceinline__ void q4_expand32(const uint4& c, uint32_t s01, char* row, int chunk0,
                                            int r, bool flip) {
  const uint32_t w[4] = {flip ? c.z : c.x, flip ? c.w : c.y, flip ? c.x : c.z, flip ? c.y : c.w};
  const uint32_t lo = (s01 & 0xff) * 0x00800080u, hi = (s01 >> 8) * 0x00800080u;
  const uint32_t s[2] = {flip ? hi : lo, flip ? lo : hi};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h[4];
    q4_unpack8(w[i], h);
#pragma unroll
    for (int x = 0; x < 4; ++x) h[x] = q4_mul2(h[x], s[i >> 1]);
    *reinterpret_cast<uint4*>(row + ((chunk0 + i) ^ (flip ? r ^ 2 : r)) * 16) =
        make_uint4(h[0], h[1], h[2], h[3]);
  }
}

// 16 consecutive TMEM columns of this thread's lane (warp-collective).
__device__ __forceinline__ void q4_tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// The MMA issuer (whole warp, one elected lane issues).  Step j, tile i: once
// softmax has written P_i(j - 1), half by half, O_i += P_i(j - 1) V(j - 1), then
// S_i(j) into the columns that P_i was in (the products run in issue order).
template <int D>
__device__ __forceinline__ void q4_tc_mma(Q4TcBars* bars, uint32_t tmem, uint32_t smem, int nq,
                                          int nt, volatile int* abort_flag) {
  using L = Q4TcLayout<D>;
  constexpr uint32_t kIdS = tc::idesc_f16(kTcRows, 128, 0, 0);
  constexpr uint32_t kIdPV = tc::idesc_f16(kTcRows, D, 0, 1);
  const uint64_t q_desc0 = tc::sdesc_sw128(smem + L::kQOff, 16, 1024);
  const uint64_t k_desc0 = tc::sdesc_sw128(smem + L::kKOff, 16, L::kGroupBytes);
  const uint64_t v_desc0 = tc::sdesc_sw128(smem + L::kVOff, 1024, L::kGroupBytes);
  bool ok = tc::mbar_wait_warp(&bars->q_full, 0, abort_flag);
  for (int j = 0; ok && j <= nt; ++j) {
    const bool has_s = j < nt, has_pv = j > 0;
    const int sk = j % kQ4TcSlots, sv = (j + kQ4TcSlots - 1) % kQ4TcSlots;
    if (has_pv &&
        !(ok = tc::mbar_wait_warp(&bars->v_full[sv], ((j - 1) / kQ4TcSlots) & 1, abort_flag)))
      break;
    const uint64_t kd = k_desc0 + (uint64_t)((sk * L::kSlotBytes) >> 4);
    const uint64_t vd = v_desc0 + (uint64_t)((sv * L::kSlotBytes) >> 4);
    for (int i = 0; i < nq; ++i) {
      const uint32_t d_o = tmem + 256 + i * 128, d_s = tmem + i * 128;
      if (has_pv) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (!(ok = tc::mbar_wait_warp(&bars->p_full[i][hf], (j - 1) & 1, abort_flag))) break;
          tc::fence_after_sync();
#pragma unroll
          for (int k = 4 * hf; k < 4 * hf + 4; ++k)
            tc::mma_ts_warp(d_o, d_s + k * 8, vd + (uint64_t)((2 * k * L::kGroupBytes) >> 4), kIdPV,
                            j > 1 || k > 0 ? 1u : 0u);
        }
        if (!ok) break;
        tc::mma_commit_warp(&bars->o_full[i]);
      }
      if (has_s) {
        if (i == 0) {
          if (!(ok = tc::mbar_wait_warp(&bars->k_full[sk], (j / kQ4TcSlots) & 1, abort_flag))) break;
          tc::fence_after_sync();
        }
        const uint64_t qd = q_desc0 + (uint64_t)((i * L::kHalves * L::kHalfBytes) >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_ss_warp(d_s, qd + (uint64_t)((((k >> 2) * L::kHalfBytes) + (k & 3) * 32) >> 4),
                          kd + (uint64_t)((((k >> 2) * 1024) + (k & 3) * 32) >> 4), kIdS, k > 0);
        tc::mma_commit_warp(&bars->s_full[i]);
      }
    }
    if (!ok) break;
    if (has_pv) tc::mma_commit_warp(&bars->v_empty[sv]);
    if (has_s) tc::mma_commit_warp(&bars->k_empty[sk]);
  }
  // every product issued so far has completed before TMEM is freed
  tc::mma_commit_warp(&bars->done);
  const uint64_t t0 = tc::globaltimer_ns();
  while (!tc::mbar_try_wait(&bars->done, 0) && tc::globaltimer_ns() - t0 < tc::kWaitLimitNs) {
  }
}

template <int D, bool ROUTED>
__global__ void __launch_bounds__(kQ4TcThreads, 1) q4_attend_tc_kernel(const Q4AttendArgs g) {
  using L = Q4TcLayout<D>;
  extern __shared__ __align__(1024) char smem_raw[];
  char* smem = reinterpret_cast<char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Q4TcBars* bars = reinterpret_cast<Q4TcBars*>(smem + L::kBarOff);
  int* ents = reinterpret_cast<int*>(smem + L::kEntOff);
  int* flags = ents + 64;
  volatile int* abort_flag = &bars->abort;
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the last rows of a sequence attend the most tokens: they start first
  const int tile = g.n_tiles - 1 - (int)blockIdx.x / g.n_split;
  const int split = blockIdx.x % g.n_split;
  const int h = blockIdx.y;
  const int z = blockIdx.z + (ROUTED ? g.z0 : 0);
  Q4Unit u;
  if (!q4_unit(g, ROUTED, z, &u)) return;
  const int G = g.a.G, nrows = u.n * G, row0 = tile * kQ4TcRows;
  if (row0 >= nrows) return;
  const int nq = nrows - row0 > kTcRows ? 2 : 1;
  const int first_pos = u.pos0 + row0 / G;
  const int last_pos = u.pos0 + min(nrows - 1, row0 + kQ4TcRows - 1) / G;

  if (warp >= 8) {
    // q's row on its way into L2 while the block sets up
    const int ur = row0 + tid - 256;
    if (ur < nrows) {
      const char* src = reinterpret_cast<const char*>(
          static_cast<const __nv_bfloat16*>(g.a.q) +
          ((u.tok0 + ur / G) * g.a.Hq + (int64_t)h * G + ur % G) * D);
#pragma unroll
      for (int x = 0; x < D * 2; x += 128) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(src + x));
    }
  }
  if (tid == 0) {
    bars->abort = 0;
    tc::mbar_init(&bars->q_full, nq * 4);
    for (int s = 0; s < kQ4TcSlots; ++s) {
      tc::mbar_init(&bars->k_full[s], kQ4TcExpand / 32);
      tc::mbar_init(&bars->v_full[s], kQ4TcExpand / 32);
      tc::mbar_init(&bars->k_empty[s], 1);
      tc::mbar_init(&bars->v_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars->s_full[i], 1);
      tc::mbar_init(&bars->o_full[i], 1);
      for (int x = 0; x < 2; ++x) tc::mbar_init(&bars->p_full[i][x], 4);
    }
    tc::mbar_init(&bars->done, 1);
    for (int s = 0; s < L::kStages; ++s) {
      tc::mbar_init(&bars->raw_full[s], 1);
      tc::mbar_init(&bars->raw_empty[s], kQ4TcExpand / 32);
    }
    tc::fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(&bars->tmem_base, 512);
    tc::tmem_relinquish();
  }
  const Q4List list = q4_list<ROUTED>(g, u, z, h, first_pos, last_pos);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  int t_lo, t_hi;
  q4_split_range((list.n + 15) / 16, g.n_split, split, &t_lo, &t_hi);
  const int nt = t_hi - t_lo;               // steps of this CTA

  if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kQ4TcOtherRegs));
    if (warp == 0 && nt > 0) {
      // ---------------------------------------------------------- MMA issuer
      q4_tc_mma<D>(bars, tmem, tc::smem_addr(smem), nq, nt, abort_flag);
    } else if (warp == 1 || warp == 2) {
      // ---------------------------------------------------------- fetch
      // Load n is half n % 2 (8 records) of step n / 2.  Lane e < 8 owns record
      // e; the places of a warp's next load are looked up one load ahead.
      const int32_t* pages = g.c.table + (int64_t)max(u.row, 0) * g.c.row_pages;
      int last_use[L::kStages];
#pragma unroll
      for (int s = 0; s < L::kStages; ++s) last_use[s] = -1;
      int ent = -1, page = -1, in = 0;
      auto look = [&](int n) {
        ent = lane < 8 && n < 2 * nt ? q4_entry<ROUTED>(list, t_lo * 16 + n * 8 + lane) : -1;
        if (ent >= 0) page = q4_page_of(g.c, pages, ent, &in);
      };
      bool gave_up = false;
      look(warp - 1);
      for (int n = warp - 1; n < 2 * nt; n += 2) {
        const int s = n % L::kStages, u_s = n / L::kStages;
        if (n >= L::kStages &&
            (gave_up = !tc::mbar_wait_warp(&bars->raw_empty[s], (u_s - 1) & 1, abort_flag)))
          break;
        // entries of the load for the masks, eight loads (four steps) deep: the
        // slot was read by the softmax of step j - 4, which is done once the
        // first half of step j - 2 is expanded (that waits for the slots of
        // step j - 4)
        const int64_t at = ent >= 0 ? q4_offset(g.c, h, page, in, q4_record_bytes(D)) : -1;
        const unsigned live = __ballot_sync(0xffffffffu, at >= 0);
        if (lane < 8) ents[(n & 7) * 8 + lane] = at >= 0 ? ent : -1;
        if (lane == 0) flags[n & 7] = live != 0xffu;
        q4_fetch8(smem + L::kRawOff + s * L::kRaw, g.c.base, at, q4_record_bytes(D), &bars->raw_full[s],
                  lane);
#pragma unroll
        for (int x = 0; x < L::kStages; ++x)
          if (x == s) last_use[x] = u_s;
        look(n + 2);
      }
      // no copy may still be landing when the block's memory goes: a stage's
      // last load is waited for (a stage that the other warp filled again was
      // waited for by the expanding warps; a block that gives up waits for what
      // this warp issued, or for the limit)
      if (lane == 0) {
#pragma unroll
        for (int x = 0; x < L::kStages; ++x) {
          if (last_use[x] < 0) continue;
          if (!gave_up && last_use[x] * L::kStages + x < 2 * nt - L::kStages) continue;
          const uint64_t t0 = tc::globaltimer_ns();
          while (!tc::mbar_try_wait(&bars->raw_full[x], last_use[x] & 1) &&
                 tc::globaltimer_ns() - t0 < tc::kWaitLimitNs) {
          }
        }
      }
    } else if (warp >= 4) {
      // ---------------------------------------------------------- expand
      // Thread (row r of a record, chunk c of 32 values), chunks first: a warp's
      // 16-byte reads are contiguous, and its writes meet every bank group once
      // a phase of 8 threads.
      constexpr int kChunks = D / 32;
      constexpr int kRec = q4_record_bytes(D);
      constexpr int kItems = 8 * 8 * kChunks / kQ4TcExpand;   // of K in a load, and of V
      const int item = tid - 128;
      const int c = item % kChunks, r = item / kChunks % 8, e0 = item / (8 * kChunks);
      constexpr int kStep = kQ4TcExpand / (8 * kChunks);       // records between a thread's items
      const bool flip = c >= 2;
      int rs = 0, ru = 0;
      for (int n = 0; n < 2 * nt; ++n) {
        if (!tc::mbar_wait_warp(&bars->raw_full[rs], ru & 1, abort_flag)) break;
        const char* raw = smem + L::kRawOff + rs * L::kRaw;
        uint4 code[2][kItems];
        uint32_t sc[2][kItems];
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          const int e = e0 + i * kStep;
          const char* at = raw + e * kRec;
          const int ent = ents[(n & 7) * 8 + e];
          const bool live = ent >= 0 && ent * 8 + r <= last_pos;
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            code[v][i] = *reinterpret_cast<const uint4*>(at + v * 4 * D + r * (D / 2) + c * 16);
            const uint32_t x = *reinterpret_cast<const unsigned short*>(at + 8 * D + v * (D / 2) +
                                                                        r * (D / 16) + c * 2);
            sc[v][i] = live ? x : 0;
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->raw_empty[rs]);
        if (++rs == L::kStages) rs = 0, ++ru;
        const int j = n >> 1, s = j % kQ4TcSlots;
        const uint32_t freed = (j / kQ4TcSlots - 1) & 1;
        bool ok = true;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          if ((n & 1) == 0 && j >= kQ4TcSlots &&
              !(ok = tc::mbar_wait_warp(v ? &bars->v_empty[s] : &bars->k_empty[s], freed, abort_flag)))
            break;
          char* base = smem + (v ? L::kVOff : L::kKOff) + s * L::kSlotBytes;
#pragma unroll
          for (int i = 0; i < kItems; ++i) {
            const int e = (n & 1) * 8 + e0 + i * kStep;
            char* row = base + e * L::kGroupBytes + (c >> 1) * 1024 + r * 128;
            q4_expand32(code[v][i], sc[v][i], row, (c & 1) * 4, r, flip);
          }
          if (n & 1) {
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(v ? &bars->v_full[s] : &bars->k_full[s]);
          }
        }
        if (!ok) break;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kQ4TcSoftmaxRegs));
    // ------------------------------------------------------------ softmax
    const int i = (warp - 8) >> 2;              // Q tile
    const int quarter = warp & 3;               // TMEM lane quarter
    const int r = quarter * 32 + lane;          // row within the Q tile
    const int unit_row = row0 + i * kTcRows + r;
    const bool row_live = unit_row < nrows;
    const int pos = u.pos0 + (row_live ? unit_row / G : 0);
    const int64_t orow =
        (u.tok0 + (row_live ? unit_row / G : 0)) * g.a.Hq + (int64_t)h * G + unit_row % G;
    const uint32_t t_row = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t t_s = t_row + i * 128, t_o = t_row + 256 + i * 128;
    float sc = 1.f;                             // log2 units of a score
    if (i < nq && nt > 0) {
      // q's rows as fp16 relative to a power of two, in the operand layout: a
      // warp brings its 32 rows in together, then each lane scales its own
      constexpr int kLanes = D / 8, kAt = 32 / kLanes;    // lanes of a row, rows at a time
      char* rows = smem + L::kQOff + i * L::kHalves * L::kHalfBytes;
      auto chunk = [&](int rr, int x) {                   // 16 bytes of a row
        return reinterpret_cast<uint4*>(rows + (x >> 3) * L::kHalfBytes + rr * 128 +
                                        (((x & 7) ^ (rr & 7)) * 16));
      };
      const int x = lane % kLanes;
      uint4 raw[kLanes];
#pragma unroll
      for (int it = 0; it < kLanes; ++it) {
        const int rr = it * kAt + lane / kLanes;
        const int64_t at = __shfl_sync(0xffffffffu, orow, rr);
        raw[it] = make_uint4(0, 0, 0, 0);
        if (unit_row - lane + rr < nrows)
          raw[it] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(g.a.q) + at * D +
                                                    x * 8);
      }
#pragma unroll
      for (int it = 0; it < kLanes; ++it)
        *chunk(quarter * 32 + it * kAt + lane / kLanes, x) = raw[it];
      __syncwarp();
      uint32_t top = 0;
#pragma unroll 4
      for (int y = 0; y < kLanes; ++y) {
        const uint4 v = *chunk(r, y);
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                     __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
      }
      top = max(top & 0xffffu, top >> 16);
      int ex = (int)(top >> 7);
      ex = top == 0 ? 127 : min(max(ex, 1), 253);
      // a row with an infinity or NaN becomes NaN, as its softmax is
      const float down = __uint_as_float(top >= 0x7f80u ? 0x7fffffffu : (uint32_t)(254 - ex) << 23);
      sc = __uint_as_float((uint32_t)ex << 23) * g.a.scale_log2;
#pragma unroll 4
      for (int y = 0; y < kLanes; ++y) {
        const uint4 in = *chunk(r, y);
        const uint32_t v[4] = {in.x, in.y, in.z, in.w};
        uint32_t o[4];
#pragma unroll
        for (int w = 0; w < 4; ++w)
          o[w] = tc::pack_half2(__uint_as_float(v[w] << 16) * down,
                                __uint_as_float(v[w] & 0xffff0000u) * down);
        *chunk(r, y) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->q_full);
    }
    float m = -INFINITY, l = 0.f;               // m: a score, not scaled
    bool ok = i < nq;
    for (int j = 0; ok && j < nt; ++j) {
      if (!(ok = tc::mbar_wait_warp(&bars->s_full[i], j & 1, abort_flag))) break;
      tc::fence_after_sync();
      uint32_t sr[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::tmem_ld32(t_s + c * 32, sr + c * 32);
      tc::tmem_wait_ld();
      if (flags[2 * j & 7] || flags[(2 * j + 1) & 7] || (t_lo + j + 1) * 16 > list.n_whole) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int ent = ents[((2 * j & 7) * 8 + e) & 63];
          const int lim = ent < 0 ? -1 : pos - ent * 8;      // columns c <= lim count
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c > lim) sr[e * 8 + c] = __float_as_uint(-INFINITY);
        }
      }
      float mx8[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) mx8[x] = -INFINITY;
#pragma unroll
      for (int c = 0; c < 128; c += 2)
        mx8[(c >> 1) & 7] = tc::fmax3(mx8[(c >> 1) & 7], __uint_as_float(sr[c]),
                                      __uint_as_float(sr[c + 1]));
      const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                             fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
      const float m_new = fmaxf(m, mx);
      float corr = 1.f;
      if (m == -INFINITY) {
        m = m_new;                              // nothing accumulated yet (O and l are zero)
      } else if ((m_new - m) * sc > kTcRescaleLog2) {
        corr = tc::ex2((m - m_new) * sc);
        m = m_new;
      }
      if (__any_sync(0xffffffffu, corr != 1.f)) {
        // O holds the products of steps < j: wait for the last one, then scale
        if (!(ok = tc::mbar_wait_warp(&bars->o_full[i], (j - 1) & 1, abort_flag))) break;
        tc::fence_after_sync();
        l *= corr;
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t orr[16];
          q4_tmem_ld16(t_o + c * 16, orr);
          tc::tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 16; ++q) orr[q] = __float_as_uint(__uint_as_float(orr[q]) * corr);
          tc::tmem_st16(t_o + c * 16, orr);
        }
      }
      const float use = m == -INFINITY ? 0.f : m;
      float neg = fmaf(-use, sc, kQ4TcShift);
      if (__any_sync(0xffffffffu, !(fabsf(neg) <= 1048576.f))) {
        // scores so large that the rounding of the product would matter: the
        // difference is taken first
#pragma unroll
        for (int c = 0; c < 128; ++c) sr[c] = __float_as_uint(__uint_as_float(sr[c]) - use);
        neg = kQ4TcShift;
      }
      const uint64_t scale2 = tc::pk2(sc, sc), neg2 = tc::pk2(neg, neg);
      uint64_t sum2[2] = {tc::pk2(0.f, 0.f), tc::pk2(0.f, 0.f)};
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t pk[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const int c = hf * 64 + 2 * x;
          const uint64_t x2 = tc::ffma2(
              tc::pk2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), scale2, neg2);
          uint64_t p2;
          if ((x & 7) >= 6) {
            p2 = tc::exp2_fma2(x2);
          } else {
            float x0, x1;
            tc::unpk2(x2, x0, x1);
            p2 = tc::pk2(tc::ex2(x0), tc::ex2(x1));
          }
          sum2[x & 1] = tc::fadd2(sum2[x & 1], p2);
          float p0, p1;
          tc::unpk2(p2, p0, p1);
          pk[x] = tc::pack_half2(p0, p1);
        }
        tc::tmem_st32(t_s + hf * 32, pk);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->p_full[i][hf]);
      }
      float a0, a1, b0, b1;
      tc::unpk2(sum2[0], a0, a1);
      tc::unpk2(sum2[1], b0, b1);
      l += (a0 + a1) + (b0 + b1);
    }
    // ---- epilogue
    if (ok && nt > 0) {
      ok = tc::mbar_wait_warp(&bars->o_full[i], (nt - 1) & 1, abort_flag);
      tc::fence_after_sync();
      // no token: the polynomial's 2^-125 are not weights (NaN scores leave m too,
      // but l is NaN then: no record's first token is a polynomial's column)
      if (m == -INFINITY && l == l) l = 0.f;
    }
    if (ok && (g.n_split == 1 || nt > 0 || split == 0)) {
      const int64_t unit = ((int64_t)blockIdx.z * gridDim.y + h) * g.n_tiles + tile;
      const int64_t part = (unit * g.n_split + split) * kQ4TcRows + i * kTcRows + r;
      const float inv = q4_inverse(l);
      // 128 bytes of each of the warp's rows at a time through shared memory
      // (this tile's Q, which no product reads any more), so that a store
      // covers whole rows' pieces.
      char* stage = smem + L::kQOff + i * L::kHalves * L::kHalfBytes + quarter * 4096;
      const bool parts = g.n_split > 1;
      auto put = [&](int chunk, uint4 v) {
        *reinterpret_cast<uint4*>(stage + lane * 128 + ((chunk ^ (lane & 7)) * 16)) = v;
      };
      auto flush = [&](int piece) {
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int rr = 4 * k + (lane >> 3), ch = lane & 7;
          const int64_t at = __shfl_sync(0xffffffffu, orow, rr);
          const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((ch ^ (rr & 7)) * 16));
          char* dst = parts ? reinterpret_cast<char*>(g.part_o + (part - lane + rr) * D)
                            : reinterpret_cast<char*>(static_cast<__nv_bfloat16*>(g.a.o) + at * D);
          if (unit_row - lane + rr < nrows) *reinterpret_cast<uint4*>(dst + piece * 128 + ch * 16) = v;
        }
        __syncwarp();
      };
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t orr[32];
        if (nt > 0) {
          tc::tmem_ld32(t_o + c * 32, orr);
          tc::tmem_wait_ld();
        } else {
#pragma unroll
          for (int q = 0; q < 32; ++q) orr[q] = 0;
        }
        if (parts) {
#pragma unroll
          for (int q = 0; q < 8; ++q) put(q, make_uint4(orr[4 * q], orr[4 * q + 1], orr[4 * q + 2], orr[4 * q + 3]));
          flush(c);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              w[x] = tc::pack_bf162(__uint_as_float(orr[8 * q + 2 * x]) * inv,
                                    __uint_as_float(orr[8 * q + 2 * x + 1]) * inv);
            put((c & 1) * 4 + q, make_uint4(w[0], w[1], w[2], w[3]));
          }
          if (c & 1) flush(c >> 1);
        }
      }
      if (row_live) {
        const float M = m * sc;
        if (q4_nonfinite(M, l)) report(HGA_ERR_DEVICE_CHECK);
        if (g.n_split > 1) g.part_ml[part] = make_float2(M, l);
        else if (g.a.lse) g.a.lse[orow] = q4_lse(M, l, kQ4TcShift);
      }
    }
  }
  griddep_launch();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

}  // namespace hga
