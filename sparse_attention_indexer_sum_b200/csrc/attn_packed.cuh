// attn_packed.cuh -- sparse attention over a paged cache of packed latent rows (included by
// attn.cu, inside its namespace; same items, split and merge as attn_mla_kernel).
//
// A row is 400 bytes (512 e2m1 codes, 16 e8m0 scales, one per 32 dims, 64 bf16 rope dims)
// or 656 (512 e4m3 codes, 4 fp32 scales, one per 128 dims, the same rope dims).  Gathering
// it moves a third or a half of a bf16 row's bytes, so what bounds this kernel is no longer
// the gather but turning codes into operands of the warp-level MMA and moving those through
// shared memory:
//   * producer warps copy the raw rows with 16-byte cp.async (a row needs 25 or 41; a warp
//     takes a whole tile of 32 rows); rows without an entry become zeros;
//   * the eight consumer warps form two groups that take an item's tiles in turn, each with
//     its own softmax state and O: one group's products fill the other's waits;
//   * a warp owns 128 latent dims (and 16 rope dims) of its group's tile in QK and in PV.
//     It expands its codes once, in registers: a lane takes 32 dims, which share one scale,
//     of four keys with 16-byte loads (the contraction's order of dims is free, Q's
//     fragments are loaded in the same order).  For PV the expanded registers are turned by
//     movmatrix into operands with the keys along K: nothing of V goes back to shared
//     memory;
//   * the quarters' partial scores meet in shared memory, where the softmax of each head is
//     computed once.  Its reference point moves only when a score exceeds it by 2^8.
// 4-bit expansion: a code s e e m, its sign at bit 15 and e e m at bits 8..6, is the bf16
// number value * 2^-126 (0.5 becomes a subnormal); one AND, one multiplication (both
// shifts at once) and one AND move two codes, and a bf16 multiplication by 2^(E - 1)
// gives two exact scaled values.  e4m3 expansion: to fp32, times the scale, rounded to bf16
// (the bf16 operands are what the MMA multiplies; 4-bit rows need no such rounding).
// Probabilities are rounded to bf16 for the product with V, as in attn_mla_kernel (off by 2^-8
// of their size at most, as the bf16 output is).  Their sum is that of the unrounded ones, in
// 32 bits, as are scores and O.
//
// Measured, 4-bit rows: 3 x 341 queries of 2048 rows of 40000 (2.1 M rows, 7.3e10 flop; L2
// holds the cache) in 375 us = 195 TFLOP/s, 0.12 of the measured bf16 rate; bf16 rows take
// 392 us there in attn_mla_kernel, e4m3 rows 472 us.  64 decode queries over 64 x 200000
// rows, with the merge: 38 us (52 MB of rows, 8 us at the measured HBM rate); bf16 44 us,
// e4m3 47 us.  A tile of 32 keys costs an SM 1550 cycles; its products alone are 68 x 9
// cycles of each tensor pipe (the warp-level MMA at M = 16 heads) and its expansion 600 of
// each integer pipe, but one group's chain is twice that: by the clock, loads, expansion and
// QK 1300, storing the partials and meeting 300, softmax 360, PV 850 (its 64 transposes keep
// pace with its 32 products), waits and the item's end 400.  Without the copies it is as
// long; two groups overlap it only in part, and registers allow no third (V, O and Q take
// 164 of a thread's 216).
// Earlier forms, on the first case: expansion by the producers into bf16 rows for the bf16
// kernel's consumers 875 us; byte-permute tables and a second expansion for PV 561 us (integer
// pipe); eight warps in step with a swizzled bf16 tile for PV 638 us; that tile with two
// groups 474 us, with dim quarters 434 us, without generic addresses 401 us, without the
// barrier that its exchange between warps needed 396 us, with movmatrix instead of the tile
// 392 us, with mbarriers between the groups 390 us, and with copies that carry no predicate
// 380 us.  Slower: sixteen consumer warps (104 registers, spilled) 605 us; PV of a tile and
// QK of the next in one stretch 457 us; tiles of 16 keys, in two groups 510 us, in three (of
// 152 registers a thread) 489 us; the transposes before the softmax or between its steps
// 410-416 us.

constexpr int PK_BK = 32;                       // keys per tile
constexpr int PK_NB = PK_BK / 8;                // in blocks of eight
constexpr int PK_KL = PK_BK / 8;                // softmax: keys of a lane
constexpr int PK_GROUPS = 2;
constexpr int PK_GTHREADS = 128;                // a group: four warps, a quarter of the dims each
constexpr int PK_CONSUMERS = PK_GROUPS * PK_GTHREADS;
constexpr int PK_PROD_WARPS = 4;
constexpr int PK_THREADS = PK_CONSUMERS + 32 * PK_PROD_WARPS;
// Registers per thread after the roles part: the block starts with 168 each (64512 in
// all), the producers give up theirs above PK_PREGS and the consumers take PK_CREGS.
constexpr int PK_CREGS = 216, PK_PREGS = 72;
static_assert(PK_CONSUMERS * PK_CREGS + 32 * PK_PROD_WARPS * PK_PREGS <= 168 * PK_THREADS,
              "the split must not exceed what the block was launched with");
static_assert(PK_GROUPS == 2, "group 0 merges group 1's part of an item");
static_assert(PK_PROD_WARPS == 4 && PK_BK == 32, "whole warpgroups change registers; a lane per row");
constexpr int PK_SROW = PK_BK + 8;              // padded partial-score row (floats)
constexpr int PK_PROW = PK_BK + 8;              // padded P row (bf16)
constexpr int PK_RROW = 144;                    // padded rope row (bytes)
// What differs between the formats.
template <int FMT>
struct PackedFmt {
  static constexpr bool MX = FMT == kFmtMxf4;
  static constexpr int CODE_ROW = MX ? 256 : 512;      // bytes of a row's codes
  static constexpr int SWAP = MX ? 4 : 1;              // see PackedStage::codes
  // a stage always serves one group and one producer
  static constexpr int STAGES = MX ? 8 : 4;
  static_assert(STAGES % PK_GROUPS == 0 && STAGES % PK_PROD_WARPS == 0,
                "every use of a stage falls to one group and one producer");
  // pairs of rows that a producer's loop copies in a piece: all 16 of a 4-bit tile (with 4:
  // 385 instead of 375 us on 3 x 341 queries), 4 of an e4m3 tile, whose rows take more
  // instructions and spill more registers otherwise (68 instead of 40 bytes; 16: 479 instead
  // of 472 us)
  static constexpr int COPY_PAIRS = MX ? 16 : 4;
  // The register that holds dim d (0..7) of the eight dims i of a lane's 32, among v[n] or
  // o, and its half: the pairs are (0, 4), (1, 5), .. as the 4-bit expansion makes them, or
  // neighbours.
  static __host__ __device__ constexpr int reg(int i, int d) {
    return 4 * i + (MX ? (d & 3) : (d >> 1));
  }
  static __host__ __device__ constexpr int half(int d) { return MX ? (d >> 2) : (d & 1); }
};
template <int FMT>
struct PackedStage {
  // 16-byte piece i of row r at place i ^ SWAP (r & 1): the 16-byte loads of two
  // neighbouring rows' four lanes then meet no bank twice
  uint8_t codes[PK_BK][PackedFmt<FMT>::CODE_ROW];
  uint8_t rope[PK_BK][PK_RROW];
  uint8_t scale[PK_BK][16];
};
struct PackedGroup {  // one consumer group's own
  alignas(16) float s_part[4][AT_H][PK_SROW];  // partial scores of the dim quarters
  alignas(16) __nv_bfloat16 p[AT_H][PK_PROW];
  float alpha[AT_H];
  float fin_m[AT_H], fin_l[AT_H];
};
template <int FMT>
struct PackedSmem {
  static constexpr int STAGES = PackedFmt<FMT>::STAGES;
  alignas(128) PackedStage<FMT> raw[STAGES];
  PackedGroup grp[PK_GROUPS];
  alignas(128) uint8_t q[AT_H][AT_ROWB];
  alignas(16) float4 o1[AT_H * AT_DV / 4];  // group 1's O at an item's end
  alignas(16) int ibuf[2][AT_MAXK];
  uint32_t vmask[STAGES];  // bit j: row j has an entry
  int last[STAGES];
  int lost[STAGES];  // the stage's group gives up: a wait ran out
  alignas(8) uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t qfull, qempty;
  uint64_t ifull[2];
  uint64_t pitem;
  uint64_t xfull, xempty;  // group 1's O and sums of an item
  int abort;
};
static_assert(sizeof(PackedSmem<kFmtMxf4>) <= 232448 && sizeof(PackedSmem<kFmtE4m3>) <= 232448,
              "shared memory of a CTA");

// 16 bytes to shared memory; with `copy`, 16 zero bytes if it is false (src is then not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool copy) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(copy ? 16 : 0)
               : "memory");
}
// An arrival on `bar` once all of this thread's earlier cp.async have landed (counted in
// the barrier's initial count).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// The copies of one tile's rows by one warp: prow is lane r's pool row of row r, or -1.
template <int FMT>
struct PackedCopy {
  uint32_t at0, at1, step;  // this lane's piece: its place in even and odd rows, the row step
  uint32_t at2 = 0, step2 = 0;  // e4m3: its other piece, of every other row
  const uint8_t *src, *src2 = nullptr;
  __device__ __forceinline__ PackedCopy(uint32_t raw0, const void* kv, int lane) {
    using S = PackedStage<FMT>;
    const uint8_t* base = static_cast<const uint8_t*>(kv);
    auto tail = [&](int i, uint32_t& at, uint32_t& st) {  // piece i behind the codes
      at = raw0 + static_cast<uint32_t>(i == 0 ? offsetof(S, scale) : offsetof(S, rope) + 16 * (i - 1));
      st = i == 0 ? 16 : PK_RROW;
    };
    src = base + 16 * lane;
    if (FMT == kFmtE4m3 || lane < 16) {
      at0 = raw0 + static_cast<uint32_t>(offsetof(S, codes)) + 16 * lane;
      at1 = raw0 + static_cast<uint32_t>(offsetof(S, codes)) + 16 * (lane ^ PackedFmt<FMT>::SWAP);
      step = PackedFmt<FMT>::CODE_ROW;
    } else {
      tail(lane - 16, at0, step);
      at1 = at0;
    }
    if constexpr (FMT == kFmtE4m3) {  // lanes 0..8: even rows, 9..17: odd rows
      const int i = lane < 9 ? lane : lane < 18 ? lane - 9 : 0;
      tail(i, at2, step2);
      if (lane >= 9) at2 += step2;
      src2 = base + 16 * (32 + i);
    }
  }
  __device__ __forceinline__ void rows(uint32_t stage_ofs, int prow, uint32_t valid, long ld,
                                       int lane) const {
    if (valid == 0xffffffffu) {  // no row is missing: the usual tile
      uint32_t d0 = at0 + stage_ofs, d1 = at1 + stage_ofs, d2 = at2 + stage_ofs;
      constexpr int kPairs = PackedFmt<FMT>::COPY_PAIRS;
#pragma unroll kPairs
      for (int r = 0; r < PK_BK; r += 2) {
        const int ra = __shfl_sync(0xffffffffu, prow, r), rb = __shfl_sync(0xffffffffu, prow, r + 1);
        if (FMT == kFmtE4m3 || lane < 25) {
          cp_async16(d0, src + static_cast<long>(ra) * ld);
          cp_async16(d1 + step, src + static_cast<long>(rb) * ld);
        }
        if constexpr (FMT == kFmtE4m3)
          if (lane < 18) cp_async16(d2, src2 + static_cast<long>(lane < 9 ? ra : rb) * ld);
        d0 += 2 * step;
        d1 += 2 * step;
        d2 += 2 * step2;
      }
      return;
    }
#pragma unroll 4
    for (int r = 0; r < PK_BK; ++r) {
      const int row = __shfl_sync(0xffffffffu, prow, r);
      const long ofs = row >= 0 ? static_cast<long>(row) * ld : 0;
      if (FMT == kFmtE4m3 || lane < 25)
        cp_async16(((r & 1) ? at1 : at0) + stage_ofs + r * step, src + ofs, row >= 0);
      if constexpr (FMT == kFmtE4m3) {
        if (r & 1) {
          const int row2 = __shfl_sync(0xffffffffu, prow, r - (lane < 9 ? 1 : 0));
          if (lane < 18)
            cp_async16(at2 + stage_ofs + (r - 1) * step2,
                       src2 + (row2 >= 0 ? static_cast<long>(row2) * ld : 0), row2 >= 0);
        }
      }
    }
  }
};

// Producers walk the items as attn_producer's do; every fourth tile is one warp's: lane l
// looks up row l of the tile, then the lanes copy the rows' 16-byte pieces.
template <int FMT>
__device__ __forceinline__ void packed_producer(PackedSmem<FMT>& sm, const AttnArgs& a,
                                                const PagedArgs& pg) {
  constexpr int STAGES = PackedFmt<FMT>::STAGES;
  const int lane = threadIdx.x & 31;
  const int pw = (threadIdx.x - PK_CONSUMERS) >> 5;
  volatile int* abort = &sm.abort;
  const bool bulk = a.idx_bulk != 0;
  const PackedCopy<FMT> copy(smem_u32(&sm.raw[0]), a.kv, lane);
  int stage = pw, ib = 0, qloads = 0;
  int t0 = pw;  // this warp's first tile of the item (its tiles of all items: every fourth)
  uint32_t ph = 0, iph[2] = {0u, 0u};
  int ipending[2] = {0, 0};
  const long nj = attn_nitems(a);
  auto load_indices = [&](long it, int b) {
    const AttnItem x = attn_item(a, it);
    const int cnt = x.end - x.beg;
    const int* src = a.idx + x.qrow * a.k + x.beg;
    if (bulk) {
      if (lane == 0) {
        const uint32_t bar = smem_u32(&sm.ifull[b]);
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(cnt) * 4u);
        if (cnt > 0) bulk_g2s(smem_u32(&sm.ibuf[b][0]), src, static_cast<uint32_t>(cnt) * 4u, bar);
      }
      ipending[b] = 1;
    } else {
      for (int j = lane; j < cnt; j += 32) sm.ibuf[b][j] = __ldg(src + j);
      __syncwarp();
    }
  };
  auto wait = [&](const uint64_t& bar, uint32_t parity) {
    return mbar_wait(smem_u32(&bar), parity, abort, kErrTimeoutProducer);
  };
  if (pw == 0 && nj > 0) load_indices(0, 0);
  for (long it = 0; it < nj; ++it, ib ^= 1) {
    const AttnItem x = attn_item(a, it);
    const int cnt = x.end - x.beg;
    const long b = x.qrow / a.R;
    const int len = min(pg.seq_lens[b], pg.max_len);
    // every producer is done with the previous item (and its index list)
    if (lane == 0) mbar_arrive(smem_u32(&sm.pitem));
    bool ok = wait(sm.pitem, static_cast<uint32_t>(it & 1));
    if (bulk) ok = ok && wait(sm.ifull[ib], iph[ib]);
    const int* ilist = sm.ibuf[ib];
    int lv = -1;  // the last entry that counts: later ones need no tiles
    for (int j = lane; j < cnt; j += 32) {
      const int s = ilist[j];
      if (s >= 0 && s < len) lv = j;
    }
    // after a wait that ran out the warp's lanes leave together, here as below
    lv = __reduce_max_sync(0xffffffffu, ok ? lv : INT_MAX);
    if (lv == INT_MAX) break;
    if (bulk) {
      iph[ib] ^= 1;
      ipending[ib] = 0;
    }
    if (pw == 0 && it + 1 < nj) load_indices(it + 1, ib ^ 1);
    const int ntiles = lv >= 0 ? lv / PK_BK + 1 : 0;
    if (pw == 0) {
      // the item's queries, once the consumers hold the previous ones in registers
      if (qloads > 0 && !__all_sync(0xffffffffu, wait(sm.qempty, (qloads - 1) & 1))) break;
      if (lane == 0) mbar_arrive_expect_tx(smem_u32(&sm.qfull), AT_H * AT_ROW_BYTES);
      __syncwarp();
      if (lane < AT_H)
        bulk_g2s(smem_u32(&sm.q[lane][0]), a.q + (x.qrow * AT_H + lane) * AT_DK, AT_ROW_BYTES,
                 smem_u32(&sm.qfull));
      ++qloads;
    }
    // the pool row of row `lane` of tile t
    auto pool_row = [&](int t) -> int {
      const int j = t * PK_BK + lane;
      const int s = (t < ntiles && j < cnt) ? ilist[j] : -1;
      if (s < 0 || s >= len) return -1;
      return static_cast<int>(attn_page_row(pg, b, s));
    };
    // the groups take turns: whole rounds of them, at least one
    const int nt = max(1, (ntiles + PK_GROUPS - 1) / PK_GROUPS) * PK_GROUPS;
    int prow = pool_row(t0);
    for (int t = t0; t < nt; t += PK_PROD_WARPS) {
      const int pnext = pool_row(t + PK_PROD_WARPS);
      const uint32_t valid = __ballot_sync(0xffffffffu, prow >= 0);
      if (!__all_sync(0xffffffffu, wait(sm.empty[stage], ph ^ 1))) {
        ok = false;
        break;
      }
      if (t < ntiles)  // a tile without entries is not looked at
        copy.rows(stage * static_cast<uint32_t>(sizeof(PackedStage<FMT>)), prow, valid, a.ld_kv,
                  lane);
      const uint32_t fb = smem_u32(&sm.full[stage]);
      cp_async_arrive(fb);
      if (lane == 0) {
        sm.vmask[stage] = valid;
        sm.last[stage] = t >= nt - PK_GROUPS;
        mbar_arrive(fb);
      }
      prow = pnext;
      stage += PK_PROD_WARPS;
      if (stage >= STAGES) {
        stage = pw;
        ph ^= 1;
      }
    }
    // the next item's first tile of this warp: the tiles of all items are dealt in turn
    t0 = (t0 - nt) & (PK_PROD_WARPS - 1);
    if (!ok) break;
  }
  // no copy is in flight when the CTA ends
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (*abort) {
    volatile int never = 0;
    if (qloads > 0) (void)mbar_wait(smem_u32(&sm.qfull), (qloads - 1) & 1, &never, kErrTimeoutDrain);
    for (int b2 = 0; b2 < 2; ++b2)
      if (pw == 0 && ipending[b2])
        (void)mbar_wait(smem_u32(&sm.ifull[b2]), iph[b2], &never, kErrTimeoutDrain);
  }
}

// ---------------------------------------------------------------- codes to bf16
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The eight codes of w (code i in bits 4i..4i+3), times the scale pair s (both halves
// 2^(E - 1)), as the bf16 pairs (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ void e2m1_expand(uint32_t w, uint32_t s, uint32_t* o) {
  const uint32_t w8 = w >> 8;
  constexpr uint32_t kMask = 0x81C081C0u;  // bits 15 and 8..6 of each half
  o[0] = bf16x2_mul(((w & 0x000F000Fu) * 0x1040u) & kMask, s);
  o[1] = bf16x2_mul(((w & 0x00F000F0u) * 0x0104u) & kMask, s);
  o[2] = bf16x2_mul(((w8 & 0x000F000Fu) * 0x1040u) & kMask, s);
  o[3] = bf16x2_mul(((w8 & 0x00F000F0u) * 0x0104u) & kMask, s);
}

// Four e4m3 codes times the group's scale, rounded to bf16: the pairs (0, 1), (2, 3).
__device__ __forceinline__ void e4m3_expand(uint32_t w, float s, uint32_t* o) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(i ? w >> 16 : w & 0xFFFFu), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    o[i] = pack_bf16(f.x * s, f.y * s);
  }
}

// D = A B (mma_bf16 with nothing to add to).
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// The 8 x 8 transpose of a matrix of 16-bit values held two a lane (row lane / 4).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Expands the codes of this warp's quarter of a tile in v and multiplies them with Q: dims
// 128 kq..+128 and rope dims 16 kq..+16 of all keys (lane: keys g + 8n, dims 32 cq..+32 of
// the quarter).  In v[n][4i] (and v[n][4i + 2] for e4m3) come the codes of dims 8i..8i+7,
// which become the four pairs v[n][4i..4i+3] (PackedFmt::reg).  The partial scores go to sp,
// the quarter's rows of heads.  e[n]: key g + 8n's scale: the block's code (4-bit), or the
// group's fp32 scale as bits.  BIG (4-bit): some scale code of the warp is above 128, so that
// 2^(E - 1) is no bf16 and the factor goes in two steps.
template <int FMT, bool BIG>
__device__ __forceinline__ void packed_qk(const PackedStage<FMT>& raw, const uint32_t (&qa)[9][4],
                                          int kq, int lane, const uint32_t (&e)[PK_NB], float* sp,
                                          uint32_t (&v)[PK_NB][16]) {
  const int g = lane >> 2, cq = lane & 3;
  float c[PK_NB][4];
  uint32_t s[PK_NB], s2[PK_NB];
  if constexpr (FMT == kFmtMxf4) {
#pragma unroll
    for (int n = 0; n < PK_NB; ++n) {
      s[n] = ((BIG && e[n] > 128u ? 128u : e[n]) + 126u) * 0x00800080u;
      if constexpr (BIG)  // the rest of larger scales: 2^(E - 128), or NaN
        s2[n] = e[n] == 255u ? 0x7FFF7FFFu
                             : ((e[n] > 128u ? e[n] - 128u : 0u) + 127u) * 0x00800080u;
    }
  }
  auto expand = [&](int n, int i) {
    if constexpr (FMT == kFmtE4m3) {
      const uint32_t w = v[n][4 * i + 2];
      e4m3_expand(v[n][4 * i], __uint_as_float(e[n]), &v[n][4 * i]);
      e4m3_expand(w, __uint_as_float(e[n]), &v[n][4 * i + 2]);
    } else {
      e2m1_expand(v[n][4 * i], s[n], &v[n][4 * i]);
      if constexpr (BIG) {
#pragma unroll
        for (int j = 4 * i; j < 4 * i + 4; ++j) v[n][j] = bf16x2_mul(v[n][j], s2[n]);
      }
    }
  };
  auto product = [&](int n, int k) {  // k: the step of 16 dims
    mma_bf16(c[n], qa[k], v[n][2 * k], v[n][2 * k + 1]);
  };
  const uint32_t rope = smem_u32(&raw.rope[(lane & 7) + 8 * (lane >> 4)][0]) + 32 * kq +
                        16 * ((lane >> 3) & 1);
#pragma unroll
  for (int n = 0; n < PK_NB; n += 2) {
    uint32_t b0, b1, b2, b3;
    ldsm_x4(rope + 8 * n * PK_RROW, b0, b1, b2, b3);
    mma_bf16_first(c[n], qa[8], b0, b1);
    mma_bf16_first(c[n + 1], qa[8], b2, b3);
  }
#pragma unroll
  for (int n = 0; n < PK_NB; ++n) expand(n, 0);
  // the products of a word run while the next word's codes are expanded
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int n = 0; n < PK_NB; ++n) {
      if (i < 3) expand(n, i + 1);
      product((2 * n) % PK_NB, 2 * i + 2 * n / PK_NB);
      product((2 * n + 1) % PK_NB, 2 * i + 2 * n / PK_NB);
    }
  float* p = sp + 2 * cq;
#pragma unroll
  for (int n = 0; n < PK_NB; ++n) {
    *reinterpret_cast<float2*>(p + g * PK_SROW + 8 * n) = make_float2(c[n][0], c[n][1]);
    *reinterpret_cast<float2*>(p + (g + 8) * PK_SROW + 8 * n) = make_float2(c[n][2], c[n][3]);
  }
}

// O = alpha O + P V for this warp's dims: a transposed register of v holds, in lane
// (g', c'), keys 2c', 2c' + 1 of column g' -- just what the MMA takes as its B operand, the
// columns being the pairs of the four lanes' blocks.
__device__ __forceinline__ void packed_pv(const uint32_t (&v)[PK_NB][16], uint32_t pbase, float al0,
                                       float al1, int lane, float (&o)[16][4]) {
  // most tiles do not move any reference point
  if (!__all_sync(0xffffffffu, al0 == 1.f && al1 == 1.f)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      o[i][0] *= al0;
      o[i][1] *= al0;
      o[i][2] *= al1;
      o[i][3] *= al1;
    }
  }
  const int pr = (lane & 7) + 8 * ((lane >> 3) & 1);
  uint32_t pa[PK_BK / 16][4];
#pragma unroll
  for (int ks = 0; ks < PK_BK / 16; ++ks)
    ldsm_x4(pbase + (pr * PK_PROW + 16 * ks + 8 * (lane >> 4)) * 2, pa[ks][0], pa[ks][1], pa[ks][2],
            pa[ks][3]);
  constexpr int kAhead = 3;  // transposes in flight ahead of their product
  uint32_t t[kAhead][2];
  auto fetch = [&](int k) {  // k: 16 ks + j
    t[k % kAhead][0] = transpose8x8(v[2 * (k >> 4)][k & 15]);
    t[k % kAhead][1] = transpose8x8(v[2 * (k >> 4) + 1][k & 15]);
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) fetch(k);
#pragma unroll
  for (int k = 0; k < PK_BK; ++k) {
    mma_bf16(o[k & 15], pa[k >> 4], t[k % kAhead][0], t[k % kAhead][1]);
    if (k + kAhead < PK_BK) fetch(k + kAhead);
  }
}

// The two groups take the tiles of an item in turn (group j those with index j mod 2) and
// keep their own softmax state and O: while one waits for its softmax or barriers, the
// other's products run.  At the item's end group 1 leaves its O in shared memory (and goes
// on), group 0 merges and stores.
template <int FMT>
__device__ __forceinline__ void packed_consumer(PackedSmem<FMT>& sm, const AttnArgs& a) {
  using F = PackedFmt<FMT>;
  const int grp = threadIdx.x / PK_GTHREADS, tid = threadIdx.x % PK_GTHREADS;
  const int warp = tid >> 5, lane = tid & 31;
  PackedGroup& G = sm.grp[grp];
  volatile int* abort = &sm.abort;
  const int g = lane >> 2, cq = lane & 3;
  const int sh = 4 * warp + (lane >> 3);  // softmax: head of this lane
  const int sk = PK_KL * (lane & 7);      // and its keys
  const uint32_t pbase = smem_u32(&G.p[0][0]);
  int stage = grp;
  uint32_t ph = 0;
  // Where a wait ran out (ok is false), the group's warps meet at the first barrier of the
  // tile at hand, or of the next one, and leave together: none is left in a barrier.
  // Each lane polls a barrier, the clock and the abort flag by itself, so at the limit some
  // lanes can have seen the barrier and others not: the warp votes before it branches, and
  // until then lanes with either answer run the same code.  (A vote, or a __syncwarp, at the
  // waits for qfull or xempty too, which no branch follows: 385-387 instead of 375 us on
  // 3 x 341 queries.)
  bool ok = true;
  auto wait = [&](const uint64_t& bar, uint32_t parity) {
    return mbar_wait(smem_u32(&bar), parity, abort, kErrTimeoutEpilogue);
  };
  auto lost = [&](int st) { return *const_cast<volatile int*>(&sm.lost[st]) != 0; };
  const long nj = attn_nitems(a);
  for (long it = 0; it < nj; ++it) {
    const AttnItem x = attn_item(a, it);
    ok = ok && wait(sm.qfull, it & 1);
    uint32_t qa[9][4];
    // dims 128 warp + 32cq + 8i..+8 of heads g, g + 8 in the pairs of the expanded codes
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ofs = (128 * warp + 32 * cq + 8 * i) * 2;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const uint4 u = *reinterpret_cast<const uint4*>(&sm.q[g + 8 * hh][ofs]);
        if constexpr (F::MX) {
          qa[2 * i][hh] = __byte_perm(u.x, u.z, 0x5410);          // dims 0, 4
          qa[2 * i][2 + hh] = __byte_perm(u.x, u.z, 0x7632);      // 1, 5
          qa[2 * i + 1][hh] = __byte_perm(u.y, u.w, 0x5410);      // 2, 6
          qa[2 * i + 1][2 + hh] = __byte_perm(u.y, u.w, 0x7632);  // 3, 7
        } else {
          qa[2 * i][hh] = u.x;
          qa[2 * i][2 + hh] = u.y;
          qa[2 * i + 1][hh] = u.z;
          qa[2 * i + 1][2 + hh] = u.w;
        }
      }
    }
    ldsm_x4(smem_u32(&sm.q[(lane & 7) + 8 * ((lane >> 3) & 1)][0]) +
                (AT_DV + 16 * warp + 8 * (lane >> 4)) * 2,
            qa[8][0], qa[8][1], qa[8][2], qa[8][3]);
    // Q's place is given back once these loads have certainly returned: after the first
    // tile whose products used them
    bool qheld = true;
    float o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m_run = -INFINITY, l_run = 0.f;  // softmax state of head sh (its 8 lanes agree)

    bool ready = false;  // the next tile was seen to have landed
    for (bool last = false; !last;) {
      if (!__all_sync(0xffffffffu, ok && (ready || wait(sm.full[stage], ph)))) {
        *const_cast<volatile int*>(&sm.lost[stage]) = 1;
        named_bar_sync(1 + grp, PK_GTHREADS);
        return;
      }
      last = sm.last[stage] != 0;
      const uint32_t vm = sm.vmask[stage];
      uint32_t v[PK_NB][16];
      if (vm) {
        const PackedStage<FMT>& raw = sm.raw[stage];
        uint32_t e[PK_NB];
#pragma unroll
        for (int n = 0; n < PK_NB; ++n) {
          const int r = g + 8 * n, blk = 4 * warp + cq;
          auto piece = [&](int i) {
            return *reinterpret_cast<const uint4*>(&raw.codes[r][16 * (i ^ (F::SWAP * (g & 1)))]);
          };
          if constexpr (F::MX) {
            const uint4 u = piece(blk);
            v[n][0] = u.x;
            v[n][4] = u.y;
            v[n][8] = u.z;
            v[n][12] = u.w;
            e[n] = raw.scale[r][blk];
          } else {
            const uint4 u = piece(2 * blk), w = piece(2 * blk + 1);
            v[n][0] = u.x;
            v[n][2] = u.y;
            v[n][4] = u.z;
            v[n][6] = u.w;
            v[n][8] = w.x;
            v[n][10] = w.y;
            v[n][12] = w.z;
            v[n][14] = w.w;
            e[n] = *reinterpret_cast<const uint32_t*>(&raw.scale[r][4 * warp]);
          }
        }
        float* sp = &G.s_part[warp][0][0];
        uint32_t emax = e[0];
#pragma unroll
        for (int n = 1; n < PK_NB; ++n) emax = max(emax, e[n]);
        if (F::MX && __any_sync(0xffffffffu, emax > 128u))
          packed_qk<FMT, F::MX>(raw, qa, warp, lane, e, sp, v);
        else
          packed_qk<FMT, false>(raw, qa, warp, lane, e, sp, v);
      }
      // the partials are complete
      named_bar_sync(1 + grp, PK_GTHREADS);
      if (tid == 0) {
        mbar_arrive(smem_u32(&sm.empty[stage]));
        if (vm && qheld) mbar_arrive(smem_u32(&sm.qempty));
      }
      if (vm) qheld = false;
      const int st = stage;
      stage += PK_GROUPS;
      if (stage >= F::STAGES) {
        stage = grp;
        ph ^= 1;
      }
      ready = false;
      if (!vm) {
        if (lost(st)) return;
        continue;
      }
      {
        float z[PK_KL];
#pragma unroll
        for (int i = 0; i < PK_KL; i += 2) {
          float2 u = *reinterpret_cast<const float2*>(&G.s_part[0][sh][sk + i]);
#pragma unroll
          for (int qq = 1; qq < 4; ++qq) {
            const float2 w = *reinterpret_cast<const float2*>(&G.s_part[qq][sh][sk + i]);
            u.x += w.x;
            u.y += w.y;
          }
          z[i] = ((vm >> (sk + i)) & 1u) ? u.x * a.scale_log2 : -INFINITY;
          z[i + 1] = ((vm >> (sk + i + 1)) & 1u) ? u.y * a.scale_log2 : -INFINITY;
        }
        // the reference point moves only when a score exceeds it by more than 2^8 in the
        // numerators: their sums have ample room, and most tiles then need no maximum
        // over the head's lanes and no rescaling of O
        float t = z[0], al = 1.f;
#pragma unroll
        for (int i = 1; i < PK_KL; ++i) t = fmaxf(t, z[i]);
        if (__any_sync(0xffffffffu, t > m_run + 8.f)) {
#pragma unroll
          for (int off = 4; off > 0; off >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
          const float n = softmax_ref(m_run, t);
          al = (n == -INFINITY) ? 1.f : fast_exp2(m_run - n);
          l_run *= al;
          m_run = n;
        }
        const float bse = (m_run == -INFINITY) ? 0.f : m_run;
#pragma unroll
        for (int i = 0; i < PK_KL; i += 2) {  // this lane's keys' share of the sum
          const float e0 = fast_exp2(z[i] - bse), e1 = fast_exp2(z[i + 1] - bse);
          l_run += e0 + e1;
          *reinterpret_cast<uint32_t*>(&G.p[sh][sk + i]) = pack_bf16(e0, e1);
        }
        if ((lane & 7) == 0) G.alpha[sh] = al;
      }
      if (lost(st)) return;
      named_bar_sync(1 + grp, PK_GTHREADS);  // P, alpha complete
      // asked before PV, so that the answer's latency hides behind it (an item's first
      // tile is waited for)
      if (!last) ready = mbar_test(smem_u32(&sm.full[stage]), ph);
      packed_pv(v, pbase, G.alpha[g], G.alpha[g + 8], lane, o);
    }

    // ---- item epilogue
    if (qheld && tid == 0) mbar_arrive(smem_u32(&sm.qempty));
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) l_run += __shfl_xor_sync(0xffffffffu, l_run, off);
    if (grp > 0 && it > 0) ok = wait(sm.xempty, (it - 1) & 1);  // the previous item's is read
    if ((lane & 7) == 0) {
      G.fin_m[sh] = m_run;
      G.fin_l[sh] = l_run;
    }
    // this lane holds dims 128 warp + 32 cq..+32 of heads g (o[.][0..1]) and g + 8
    // (o[.][2..3]), placed as PackedFmt::reg says; group 1 leaves four floats per (j, lane)
    if (grp > 0) {
      float4* dst = sm.o1 + warp * 512 + lane;
#pragma unroll
      for (int j = 0; j < 16; ++j) dst[32 * j] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.xfull));
    } else {
      named_bar_sync(1 + grp, PK_GTHREADS);  // fin_m, fin_l of this group
      ok = __all_sync(0xffffffffu, wait(sm.xfull, it & 1));
      if (!ok) continue;
      float wt[2][2], M[2], L[2];  // the groups' weights, and their sums: heads g, g + 8
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int h = g + 8 * hh;
        M[hh] = fmaxf(sm.grp[0].fin_m[h], sm.grp[1].fin_m[h]);
        L[hh] = 0.f;
#pragma unroll
        for (int x2 = 0; x2 < 2; ++x2) {
          const float m = sm.grp[x2].fin_m[h];
          wt[x2][hh] = m == -INFINITY ? 0.f : fast_exp2(m - M[hh]);
          L[hh] += sm.grp[x2].fin_l[h] * wt[x2][hh];
        }
        if (!a.split) {
          const float inv = L[hh] > 0.f ? 1.f / L[hh] : 0.f;
          wt[0][hh] *= inv;
          wt[1][hh] *= inv;
        }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        o[j][0] *= wt[0][0];
        o[j][1] *= wt[0][0];
        o[j][2] *= wt[0][1];
        o[j][3] *= wt[0][1];
        const float4 u = sm.o1[warp * 512 + lane + 32 * j];
        o[j][0] += u.x * wt[1][0];
        o[j][1] += u.y * wt[1][0];
        o[j][2] += u.z * wt[1][1];
        o[j][3] += u.w * wt[1][1];
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int h = g + 8 * hh, d = 128 * warp + 32 * cq;
        if (!a.split) {
          uint32_t* ob = reinterpret_cast<uint32_t*>(a.out + (x.qrow * AT_H + h) * AT_DV + d);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t r[4];
#pragma unroll
            for (int b = 0; b < 4; ++b)
              r[b] = pack_bf16(o[F::reg(i, 2 * b)][2 * hh + F::half(2 * b)],
                               o[F::reg(i, 2 * b + 1)][2 * hh + F::half(2 * b + 1)]);
            if ((reinterpret_cast<uintptr_t>(a.out) & 15) == 0) {
              reinterpret_cast<uint4*>(ob)[i] = make_uint4(r[0], r[1], r[2], r[3]);
            } else {  // only required to be aligned to 4
#pragma unroll
              for (int b = 0; b < 4; ++b) ob[4 * i + b] = r[b];
            }
          }
        } else {
          float4* po = reinterpret_cast<float4*>(a.part_o + (x.pslot * AT_H + h) * AT_DV + d);
          auto at = [&](int i, int b) { return o[F::reg(i, b)][2 * hh + F::half(b)]; };
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int b = 0; b < 2; ++b)
              po[2 * i + b] = make_float4(at(i, 4 * b), at(i, 4 * b + 1), at(i, 4 * b + 2),
                                          at(i, 4 * b + 3));
        }
      }
      if (warp == 0 && cq == 0) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int h = g + 8 * hh;
          if (a.split) {
            a.part_ml[(x.pslot * AT_H + h) * 2] = M[hh];
            a.part_ml[(x.pslot * AT_H + h) * 2 + 1] = L[hh];
          } else if (a.lse) {
            a.lse[x.qrow * AT_H + h] = attn_lse(M[hh], L[hh]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.xempty));  // group 1's O and sums have been read
    }
  }
}

template <int FMT>
__global__ void __launch_bounds__(PK_THREADS, 1)
    attn_packed_kernel(const AttnArgs a, const __grid_constant__ PagedArgs pg) {
  // (not rounded up through an integer: the compiler would lose the address space and use
  // generic loads and stores: 434 us instead of 401 on 3 x 341 queries of 2048 rows)
  extern __shared__ __align__(128) uint8_t packed_smem[];
  PackedSmem<FMT>& sm = *reinterpret_cast<PackedSmem<FMT>*>(packed_smem);
  if (threadIdx.x == 0) {
    for (int s = 0; s < PackedFmt<FMT>::STAGES; ++s) {
      // the copies of one producer warp's threads, and its arrival after the flags
      mbar_init(smem_u32(&sm.full[s]), 32 + 1);
      mbar_init(smem_u32(&sm.empty[s]), 1);
      sm.lost[s] = 0;
    }
    mbar_init(smem_u32(&sm.qfull), 1);
    mbar_init(smem_u32(&sm.qempty), PK_GROUPS);
    mbar_init(smem_u32(&sm.ifull[0]), 1);
    mbar_init(smem_u32(&sm.ifull[1]), 1);
    mbar_init(smem_u32(&sm.pitem), PK_PROD_WARPS);
    mbar_init(smem_u32(&sm.xfull), PK_GTHREADS / 32);
    mbar_init(smem_u32(&sm.xempty), PK_GTHREADS / 32);
    sm.abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  grid_dep_wait();  // set-up above touches no global memory
  if (threadIdx.x >= PK_CONSUMERS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PK_PREGS));
    packed_producer(sm, a, pg);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PK_CREGS));
    packed_consumer(sm, a);
  }
  __syncthreads();
}

template <int FMT>
static ic_status launch_attn_packed(const AttnArgs& a, const PagedArgs& pg, long grid,
                                    cudaStream_t stream) {
  const int smem = static_cast<int>(sizeof(PackedSmem<FMT>));
  ic_status st = cuda_check(cudaFuncSetAttribute(attn_packed_kernel<FMT>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                            "cudaFuncSetAttribute(attn_packed)");
  if (st) return st;
  return cuda_check(launch_dep(attn_packed_kernel<FMT>, dim3(static_cast<unsigned>(grid)),
                               dim3(PK_THREADS), smem, stream, 1, a, pg),
                    "attn_packed_kernel launch");
}
