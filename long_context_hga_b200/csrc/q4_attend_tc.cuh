// Attention over the 4-bit cache with many query rows (prompts, routed blocks;
// bf16) on the sm_100a tensor cores: tcgen05.mma with TMEM accumulators.
//
// Units, query rows and entries are those of q4_attend.cuh.  A CTA takes 256
// rows of a unit as two 128-row tiles Q0/Q1 and walks its tokens in tiles of
// 128 (16 records):
//   S_i = Q_i K^T,  O_i += P_i V       (fp16 operands, fp32 accumulators)
// K and V are expanded to fp16 on their way into shared memory, where a code
// times its scale is exact, so nothing is rounded there.  Q enters as fp16
// relative to a power of two of its row (see q4_attend.cuh).
//
// Warp roles (512 threads, registers split 80 : 176):
//   warp 0       TMEM owner and MMA issuer (tc_mma_loop)
//   warps 4-7    expand: codes of the next tile are in registers (plain
//                16-byte loads, one tile ahead) while this one is converted
//                into the 128-byte swizzled operand layout; tokens past the
//                sequence and missing pages become zeros
//   warps 8-15   softmax of Q0 and Q1, one thread per row, as in attend_tc.cuh
//                (of every 16 exponentials 6 are a polynomial on the FMA pipe)
// TMEM columns: S0 [0,128) S1 [128,256) O0 [256,256+D) O1 [384,384+D).
//
// Weights are held as 2^7 exp(score - m), m the running maximum, which is only
// moved when it grows by more than 2^8 (so that O is rarely rescaled): at most
// 2^15 in fp16, with 11 bits down to 2^-21 of the largest weight.
#pragma once
#include "attend_tc.cuh"
#include "q4_attend.cuh"

namespace hga {

constexpr int kQ4TcThreads = 512;
constexpr int kQ4TcRows = 256;
constexpr int kQ4TcExpand = 128;           // threads that expand K and V
constexpr int kQ4TcEnts = kTcTok / 8;      // records of a token tile
constexpr float kQ4TcShift = 7.f;

template <int D>
struct Q4TcLayout {
  using T = TcLayout<D>;
  static constexpr int kBarOff = T::kBarOff;
  static constexpr int kEntOff = kBarOff + 512;          // [4][16] entries, [4] flags
  static constexpr int kListOff = kEntOff + 4 * kQ4TcEnts * 4 + 64;
  static constexpr size_t smem_bytes(int max_list) {
    return 1024 + (size_t)kListOff + (size_t)max_list * 4;
  }
};

// 32 codes (16 bytes) with two scale bytes -> 64 bytes of a row of the operand
// layout, as four 16-byte chunks with the row's swizzle.
__device__ __forceinline__ void q4_expand32(const uint4& c, uint32_t s01, char* row, int chunk0,
                                            int r) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  const uint32_t s[2] = {(s01 & 0xff) * 0x00800080u, (s01 >> 8) * 0x00800080u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h[4];
    q4_unpack8(w[i], h);
#pragma unroll
    for (int x = 0; x < 4; ++x) h[x] = q4_mul2(h[x], s[i >> 1]);
    *reinterpret_cast<uint4*>(row + ((chunk0 + i) ^ r) * 16) = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

template <int D, bool ROUTED>
__global__ void __launch_bounds__(kQ4TcThreads, 1) q4_attend_tc_kernel(const Q4AttendArgs g) {
  using L = TcLayout<D>;
  using LQ = Q4TcLayout<D>;
  extern __shared__ __align__(1024) char smem_raw[];
  char* smem = reinterpret_cast<char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TcBars* bars = reinterpret_cast<TcBars*>(smem + LQ::kBarOff);
  int* ents = reinterpret_cast<int*>(smem + LQ::kEntOff);
  int* flags = ents + 4 * kQ4TcEnts;
  int* list = reinterpret_cast<int*>(smem + LQ::kListOff);
  char* sQ = smem + L::kQOff;
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

  if (tid == 0) {
    bars->abort = 0;
    tc::mbar_init(&bars->q_full, nq * kTcRows);
    for (int s = 0; s < kTcSlots; ++s) {
      tc::mbar_init(&bars->full[s], kQ4TcExpand);
      tc::mbar_init(&bars->empty[s], 1);
      tc::mbar_init(&bars->v_ready[s], kQ4TcExpand);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars->s_full[i], 1);
      tc::mbar_init(&bars->p_full[i], kTcRows);
      tc::mbar_init(&bars->o_full[i], 1);
    }
    tc::mbar_init(&bars->done, 1);
    tc::fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(&bars->tmem_base, 512);
    tc::tmem_relinquish();
  }
  int n_ent = 0, n_nondiag = 0;
  if constexpr (ROUTED) {
    bool inv = false;
    const int64_t b0 = g.a.q_start + (int64_t)z * g.a.qblock;
    n_ent = build_group_list_tc(g.a, z, h, b0, u.ctx, list, &n_nondiag, &inv);
  } else if (u.row >= 0) {
    n_ent = (last_pos >> 3) + 1;
    n_nondiag = (first_pos + 1) >> 3;       // records that every row attends whole
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  int t_lo, t_hi;
  q4_split_range((n_ent + kQ4TcEnts - 1) / kQ4TcEnts, g.n_split, split, &t_lo, &t_hi);
  const int nt = t_hi - t_lo;               // token tiles of this CTA

  if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n");
    if (warp == 0 && nt > 0) {
      // ---------------------------------------------------------- MMA issuer
      tc_mma_loop<D, 0>(bars, tmem, tc::smem_addr(sQ), tc::smem_addr(smem + L::kSlotOff), nq, nt,
                          abort_flag);
    } else if (warp >= 4 && nt > 0) {
      // ---------------------------------------------------------- expand
      // Thread (row r of a record, chunk c of 32 values); a warp takes whole
      // records (D = 128) or two at a time (D = 64), so that its loads are
      // contiguous and the 8 rows of a record meet 8 different bank groups.
      constexpr int kChunks = D / 32;
      constexpr int kPer = 32 / (8 * kChunks);          // records of a warp's load
      constexpr int kItems = kQ4TcEnts / (4 * kPer);
      constexpr int kRec = q4_record_bytes(D);
      const int w = warp - 4, r = lane & 7, c = (lane >> 3) % kChunks;
      const int sub = (lane >> 3) / kChunks;
      const int32_t* pages = g.c.table + (int64_t)u.row * g.c.row_pages;
      // Lane e < 16 finds record e of a tile: its byte offset from the plane's
      // first page, -1 where there is none.
      int ent;
      auto locate = [&](int j) -> int64_t {
        const int li = (t_lo + j) * kQ4TcEnts + (lane & 15);
        ent = -1;
        if (j < nt && li < n_ent) ent = ROUTED ? list[li] : li;
        if (ent < 0) return -1;
        const int col = ent / g.c.page_recs, in = ent - col * g.c.page_recs;
        const int pg = col < g.c.row_pages ? pages[col] : -1;
        if (pg < 0 || pg >= g.c.n_pages) {
          if (lane < 16 && w == 0) report(HGA_ERR_DEVICE_CHECK);
          ent = -1;
          return -1;
        }
        return pg * g.c.page_bytes + ((int64_t)h * g.c.page_recs + in) * kRec;
      };
      // loads this thread's items of K (which = 0) or V; scales of tokens past
      // the sequence are 0
      auto load = [&](int64_t off, int e_of, int which, uint4* code, uint32_t* sc) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          const int e = (i * 4 + w) * kPer + sub;
          const int64_t at = __shfl_sync(0xffffffffu, off, e);
          const int ee = __shfl_sync(0xffffffffu, e_of, e);
          code[i] = make_uint4(0, 0, 0, 0);
          sc[i] = 0;
          if (at >= 0 && ee * 8 + r <= last_pos) {
            const char* p = g.c.base + at;
            code[i] = *reinterpret_cast<const uint4*>(p + which * 4 * D + r * (D / 2) + c * 16);
            sc[i] = *reinterpret_cast<const unsigned short*>(p + 8 * D + which * (D / 2) +
                                                             r * (D / 16) + c * 2);
          }
        }
      };
      auto store = [&](int s, const uint4* code, const uint32_t* sc) {
        char* base = smem + L::kSlotOff + s * L::kSlotBytes;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          const int e = (i * 4 + w) * kPer + sub;
          char* row = base + e * L::kGroupBytes + (c >> 1) * 1024 + r * 128;
          q4_expand32(code[i], sc[i], row, (c & 1) * 4, r);
        }
        tc::fence_proxy_async_smem();
      };
      uint4 kc[kItems], vc[kItems];
      uint32_t ks[kItems], vs[kItems];
      int64_t off = locate(0);
      int e_of = ent;
      load(off, e_of, 0, kc, ks);
      load(off, e_of, 1, vc, vs);
      bool ok = true;
      for (int j = 0; j < nt; ++j) {
        if (w == 0) {
          // entries of the tile for the softmax warps' masks, four tiles deep
          const unsigned live = __ballot_sync(0xffffffffu, e_of >= 0);
          if (lane < kQ4TcEnts) ents[(j & 3) * kQ4TcEnts + lane] = e_of;
          if (lane == 0) flags[j & 3] = (live & 0xffffu) != 0xffffu;
        }
        off = locate(j + 1);
        e_of = ent;
        int n = 2 * j, s = n % kTcSlots;
        if (n >= kTcSlots &&
            !(ok = tc::mbar_wait_warp(&bars->empty[s], (n / kTcSlots - 1) & 1, abort_flag)))
          break;
        store(s, kc, ks);
        tc::mbar_arrive(&bars->full[s]);
        load(off, e_of, 0, kc, ks);
        ++n, ++s;
        if (n >= kTcSlots &&
            !(ok = tc::mbar_wait_warp(&bars->empty[s], (n / kTcSlots - 1) & 1, abort_flag)))
          break;
        store(s, vc, vs);
        tc::mbar_arrive(&bars->v_ready[s]);
        load(off, e_of, 1, vc, vs);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;\n");
    // ------------------------------------------------------------ softmax
    const int i = (warp - 8) >> 2;              // Q tile of this warpgroup
    const int quarter = warp & 3;               // TMEM lane quarter
    const int r = quarter * 32 + lane;          // row within the Q tile
    const int unit_row = row0 + i * kTcRows + r;
    const bool row_live = unit_row < nrows;
    const int pos = u.pos0 + (row_live ? unit_row / G : 0);
    const int64_t orow =
        (u.tok0 + (row_live ? unit_row / G : 0)) * g.a.Hq + (int64_t)h * G + unit_row % G;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t t_s = tmem + lane_off + i * 128;
    const uint32_t t_o = tmem + lane_off + 256 + i * 128;
    float sc = 1.f;                             // log2 units of a score
    if (i < nq && nt > 0) {
      // q's row as fp16 relative to a power of two, in the operand layout
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const __nv_bfloat16*>(g.a.q) + orow * D);
      uint4 raw[D / 8];
      uint32_t top = 0;
#pragma unroll
      for (int x = 0; x < D / 8; ++x) {
        raw[x] = row_live ? src[x] : make_uint4(0, 0, 0, 0);
        const uint32_t v[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
#pragma unroll
        for (int y = 0; y < 4; ++y) top = max(top, max(v[y] & 0x7fffu, (v[y] >> 16) & 0x7fffu));
      }
      int ex = (int)(top >> 7);
      ex = top == 0 ? 127 : min(max(ex, 1), 253);
      const float down = __uint_as_float((uint32_t)(254 - ex) << 23);
      sc = __uint_as_float((uint32_t)ex << 23) * g.a.scale_log2;
      char* row = sQ + i * L::kHalves * L::kHalfBytes + r * 128;
#pragma unroll
      for (int x = 0; x < D / 8; ++x) {
        const uint32_t v[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
        uint32_t o[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          o[y] = tc::pack_half2(__uint_as_float(v[y] << 16) * down,
                                __uint_as_float(v[y] & 0xffff0000u) * down);
        *reinterpret_cast<uint4*>(row + (x >> 3) * L::kHalfBytes + (((x & 7) ^ (r & 7)) * 16)) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
      tc::fence_proxy_async_smem();
      tc::mbar_arrive(&bars->q_full);
    }
    float m = -INFINITY, l = 0.f;               // m: a score, not scaled
    bool ok = i < nq;
    for (int j = 0; ok && j < nt; ++j) {
      if (!(ok = tc::mbar_wait_warp(&bars->s_full[i], j & 1, abort_flag))) break;
      tc::fence_after_sync();
      uint32_t sr[kTcTok];
#pragma unroll
      for (int c = 0; c < kTcTok / 32; ++c) tc::tmem_ld32(t_s + c * 32, sr + c * 32);
      tc::tmem_wait_ld();
      if (flags[j & 3] || (t_lo + j + 1) * kQ4TcEnts > n_nondiag) {
#pragma unroll
        for (int e = 0; e < kQ4TcEnts; ++e) {
          const int ent = ents[(j & 3) * kQ4TcEnts + e];
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
      for (int c = 0; c < kTcTok; c += 2)
        mx8[(c >> 1) & 7] = tc::fmax3(mx8[(c >> 1) & 7], __uint_as_float(sr[c]),
                                      __uint_as_float(sr[c + 1]));
      const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                             fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
      const float m_new = fmaxf(m, mx);
      float corr = 1.f;
      bool rescale = false;
      if (m == -INFINITY) {
        m = m_new;                              // nothing accumulated yet (O and l are zero)
        corr = 0.f;
      } else if ((m_new - m) * sc > kTcRescaleLog2) {
        corr = tc::ex2((m - m_new) * sc);
        rescale = true;
        m = m_new;
      }
      l *= corr;
      const float use = m == -INFINITY ? 0.f : m;
      float neg = fmaf(-use, sc, kQ4TcShift);
      if (__any_sync(0xffffffffu, fabsf(neg) > 1048576.f)) {
        // scores so large that the rounding of the product would matter: the
        // difference is taken first
#pragma unroll
        for (int c = 0; c < kTcTok; ++c) sr[c] = __float_as_uint(__uint_as_float(sr[c]) - use);
        neg = kQ4TcShift;
      }
      const uint64_t scale2 = tc::pk2(sc, sc);
      const uint64_t neg2 = tc::pk2(neg, neg);
      uint64_t sum2[2] = {tc::pk2(0.f, 0.f), tc::pk2(0.f, 0.f)};
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const uint64_t x2 = tc::ffma2(tc::pk2(__uint_as_float(sr[64 * hf + c]),
                                                __uint_as_float(sr[64 * hf + c + 1])),
                                       scale2, neg2);
          uint64_t p2;
          if (((c >> 1) & 7) >= 5) {
            p2 = tc::exp2_fma2(x2);
          } else {
            float x0, x1;
            tc::unpk2(x2, x0, x1);
            p2 = tc::pk2(tc::ex2(x0), tc::ex2(x1));
          }
          sum2[(c >> 1) & 1] = tc::fadd2(sum2[(c >> 1) & 1], p2);
          float p0, p1;
          tc::unpk2(p2, p0, p1);
          pk[c >> 1] = tc::pack_half2(p0, p1);
        }
        tc::tmem_st32(t_s + hf * 32, pk);
      }
      {
        float a0, a1, b0v, b1v;
        tc::unpk2(sum2[0], a0, a1);
        tc::unpk2(sum2[1], b0v, b1v);
        l += (a0 + a1) + (b0v + b1v);
      }
      if (__any_sync(0xffffffffu, rescale) && j > 0) {
        // O holds the products of tiles < j: wait for the last one, then scale
        if (!(ok = tc::mbar_wait_warp(&bars->o_full[i], (j - 1) & 1, abort_flag))) break;
        tc::fence_after_sync();
        const float f = rescale ? corr : 1.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t orr[32];
          tc::tmem_ld32(t_o + c * 32, orr);
          tc::tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 32; ++q) orr[q] = __float_as_uint(__uint_as_float(orr[q]) * f);
          tc::tmem_st32(t_o + c * 32, orr);
        }
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      tc::mbar_arrive(&bars->p_full[i]);
    }
    // ---- epilogue
    if (ok && (nt == 0 || tc::mbar_wait_warp(&bars->o_full[i], (nt - 1) & 1, abort_flag))) {
      tc::fence_after_sync();
      if (m == -INFINITY) l = 0.f;              // no token: the polynomial's 2^-125 are not weights
      const float M = m * sc;
      const int64_t unit = ((int64_t)blockIdx.z * gridDim.y + h) * g.n_tiles + tile;
      const int64_t part = (unit * g.n_split + split) * kQ4TcRows + i * kTcRows + r;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      if (g.n_split == 1 || t_lo < t_hi || split == 0) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t orr[32];
          if (nt > 0) {
            tc::tmem_ld32(t_o + c * 32, orr);
            tc::tmem_wait_ld();
          } else {
#pragma unroll
            for (int q = 0; q < 32; ++q) orr[q] = 0;
          }
          if (row_live && g.n_split > 1) {
            float4* dst = reinterpret_cast<float4*>(g.part_o + part * D + c * 32);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              dst[q] = make_float4(__uint_as_float(orr[4 * q]), __uint_as_float(orr[4 * q + 1]),
                                   __uint_as_float(orr[4 * q + 2]), __uint_as_float(orr[4 * q + 3]));
          } else if (row_live) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(g.a.o) + orow * D + c * 32);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                w[x] = tc::pack_bf162(__uint_as_float(orr[8 * q + 2 * x]) * inv,
                                      __uint_as_float(orr[8 * q + 2 * x + 1]) * inv);
              dst[q] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
        }
        if (row_live) {
          if (g.n_split > 1) g.part_ml[part] = make_float2(M, l);
          else if (g.a.lse)
            g.a.lse[orow] = l > 0.f ? (M + (log2f(l) - kQ4TcShift)) * 0.6931471805599453f : -INFINITY;
        }
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
