// attn_kv4.cuh -- sparse attention over a paged cache of 4-bit latent rows (included by
// attn.cu, inside its namespace; same items, split and merge as attn_mla_kernel).
//
// A row is 400 bytes: 512 e2m1 codes, 16 e8m0 scales (one per 32 dims), 64 bf16 rope
// dims.  Gathering it moves a third of a bf16 row's bytes, so what bounds this kernel is
// no longer the gather but turning codes into operands of the warp-level MMA:
//   * the raw rows stay as they are in shared memory (tiles of K4_BK keys, K4_STAGES
//     deep); no bf16 copy of a tile exists.  Each code is expanded twice, in the
//     registers that feed QK and in those that feed PV;
//   * QK: the contraction's order of dims is free, so lane c of a quad takes 32
//     consecutive dims -- one block, one scale -- of its key with one 16-byte load, and
//     Q's fragments are loaded in the same order;
//   * PV: a lane takes 8 consecutive dims of two keys with two 4-byte loads, and the
//     order of output dims that follows gives every lane 16 consecutive ones to store.
// Expansion: byte permutes (prmt) look up four codes at a time in a table of the eight
// magnitudes, high and low bytes of bf16 apart; QK's table is scaled beforehand, PV's
// values after.  A code times a power of two is exact in bf16.
// Rows without an entry are filled with zeros by their copies.

constexpr int K4_BK = 64;                       // keys per tile
constexpr int K4_STAGES = 4;
constexpr int K4_PROD_WARPS = 4;                // each copies 16 of a tile's 64 rows
constexpr int K4_THREADS = AT_CONSUMERS + 32 * K4_PROD_WARPS;
constexpr int K4_CHUNKS = KV4_ROW_BYTES / 16;   // 16-byte copies per row
constexpr int K4_SROW = 72;                     // padded partial-score row (floats)
constexpr int K4_PROW = 72;                     // padded P row (bf16)

struct Kv4Smem {
  alignas(128) uint8_t raw[K4_STAGES][K4_BK][KV4_ROW_BYTES];
  alignas(128) uint8_t q[AT_H][AT_ROWB];
  alignas(16) float s_part[4][AT_H][K4_SROW];
  alignas(16) __nv_bfloat16 p[AT_H][K4_PROW];
  float alpha[AT_H];
  float fin_m[AT_H], fin_l[AT_H];
  alignas(16) int ibuf[2][AT_MAXK];
  alignas(8) uint16_t vmask[K4_STAGES][4];      // bit j of [w]: row 16w + j has an entry
  int last[K4_STAGES];
  alignas(8) uint64_t full[K4_STAGES];
  uint64_t empty[K4_STAGES];
  uint64_t qfull, qempty;
  uint64_t ifull[2];
  uint64_t pitem;
  int abort;
};

// 16 bytes to shared memory, or 16 zero bytes if !copy (src is then not read).
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

// Producers walk the items as attn_producer's do; warp pw copies rows 16pw..16pw+15 of
// every tile, 25 16-byte copies each, spread over its lanes.
__device__ __forceinline__ void kv4_producer(Kv4Smem& sm, const AttnArgs& a, const PagedArgs& pg) {
  const int lane = threadIdx.x & 31;
  const int pw = (threadIdx.x - AT_CONSUMERS) >> 5;
  volatile int* abort = &sm.abort;
  const bool bulk = a.idx_bulk != 0;
  const uint8_t* kv = reinterpret_cast<const uint8_t*>(a.kv);
  const uint32_t raw0 = smem_u32(&sm.raw[0][0][0]);
  int stage = 0, ib = 0, qloads = 0;
  uint32_t ph = 0, iph[2] = {0u, 0u};
  int ipending[2] = {0, 0};
  const long nj = attn_nitems(a);
  auto load_indices = [&](long it, int b) {
    const AttnItem x = attn_item<K4_BK>(a, it);
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
  if (pw == 0 && nj > 0) load_indices(0, 0);
  for (long it = 0; it < nj; ++it, ib ^= 1) {
    const AttnItem x = attn_item<K4_BK>(a, it);
    const int cnt = x.end - x.beg;
    const long b = x.qrow / a.R;
    const int len = min(pg.seq_lens[b], pg.max_len);
    // every producer is done with the previous item (and its index list)
    if (lane == 0) mbar_arrive(smem_u32(&sm.pitem));
    if (!mbar_wait(smem_u32(&sm.pitem), static_cast<uint32_t>(it & 1), abort, kErrTimeoutProducer))
      break;
    if (pw == 0 && it + 1 < nj) load_indices(it + 1, ib ^ 1);
    if (bulk) {
      if (!mbar_wait(smem_u32(&sm.ifull[ib]), iph[ib], abort, kErrTimeoutProducer)) break;
      iph[ib] ^= 1;
      ipending[ib] = 0;
    }
    const int* ilist = sm.ibuf[ib];
    int lv = -1;  // the last entry that counts: later ones need no tiles
    for (int j = lane; j < cnt; j += 32) {
      const int s = ilist[j];
      if (s >= 0 && s < len) lv = j;
    }
    lv = __reduce_max_sync(0xffffffffu, lv);
    const int ntiles = lv >= 0 ? lv / K4_BK + 1 : 0;
    if (pw == 0) {
      // the item's queries, once the consumers hold the previous ones in registers
      if (qloads > 0 &&
          !mbar_wait(smem_u32(&sm.qempty), (qloads - 1) & 1, abort, kErrTimeoutProducer))
        break;
      if (lane == 0) mbar_arrive_expect_tx(smem_u32(&sm.qfull), AT_H * AT_ROW_BYTES);
      __syncwarp();
      if (lane < AT_H)
        bulk_g2s(smem_u32(&sm.q[lane][0]), a.q + (x.qrow * AT_H + lane) * AT_DK, AT_ROW_BYTES,
                 smem_u32(&sm.qfull));
      ++qloads;
    }
    // the pool row of row (16pw + lane mod 16) of tile t, read one tile ahead
    auto pool_row = [&](int t) -> long {
      const int j = t * K4_BK + 16 * pw + (lane & 15);
      const int s = (t < ntiles && j < cnt) ? ilist[j] : -1;
      if (!in_bounds(s >= -1 && s < len, kErrBoundsGather) || s < 0 || s >= len) return -1;
      return attn_page_row(pg, b, s);
    };
    const int nt = ntiles > 0 ? ntiles : 1;  // an empty item still ends with one (empty) tile
    long prow = pool_row(0);
    bool ok = true;
    for (int t = 0; t < nt; ++t) {
      const long pnext = pool_row(t + 1);
      if (!mbar_wait(smem_u32(&sm.empty[stage]), ph ^ 1, abort, kErrTimeoutProducer)) {
        ok = false;
        break;
      }
      const unsigned valid = __ballot_sync(0xffffffffu, prow >= 0) & 0xFFFFu;
      const uint32_t dst = raw0 + (stage * K4_BK + 16 * pw) * KV4_ROW_BYTES;
#pragma unroll
      for (int i = 0; i < (16 * K4_CHUNKS + 31) / 32; ++i) {
        const int c = lane + 32 * i;
        const int r = c / K4_CHUNKS;  // row of the warp's 16
        const long row = __shfl_sync(0xffffffffu, prow, r & 15);
        if (c < 16 * K4_CHUNKS)
          cp_async16(dst + 16 * c, kv + (row >= 0 ? row * a.ld_kv + 16 * (c - r * K4_CHUNKS) : 0),
                     row >= 0);
      }
      const uint32_t fb = smem_u32(&sm.full[stage]);
      cp_async_arrive(fb);
      if (lane == 0) {
        sm.vmask[stage][pw] = static_cast<uint16_t>(valid);
        if (pw == 0) sm.last[stage] = (t == nt - 1);
        mbar_arrive(fb);
      }
      prow = pnext;
      if (++stage == K4_STAGES) {
        stage = 0;
        ph ^= 1;
      }
    }
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
// The eight e2m1 magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 as bf16: high bytes of the first
// and last four, low bytes of the same.
struct E2m1Table {
  uint32_t h0, h1, l0, l1;
};
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The table times the power of two of e8m0 code e (0 counts as 0 instead of 2^-127, which
// no result can show; 255: zeros become NaN, as a NaN block's codes are 0).
__device__ __forceinline__ E2m1Table e2m1_table(uint32_t e) {
  const uint32_t s = e * 0x00800080u;
  const uint32_t a = bf16x2_mul(0x3F000000u, s), b = bf16x2_mul(0x3FC03F80u, s);
  const uint32_t c = bf16x2_mul(0x40404000u, s), d = bf16x2_mul(0x40C04080u, s);
  return E2m1Table{__byte_perm(a, b, 0x7531), __byte_perm(c, d, 0x7531),
                   __byte_perm(a, b, 0x6420), __byte_perm(c, d, 0x6420)};
}
// The eight codes of w (code i in bits 4i..4i+3) as four bf16 pairs (0, 1), (2, 3), ...
__device__ __forceinline__ void e2m1_expand(uint32_t w, const E2m1Table& t, uint32_t (&o)[4]) {
  const uint32_t m = w & 0x77777777u, w4 = w << 4;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t sel = half ? m >> 16 : m;
    uint32_t hi = __byte_perm(t.h0, t.h1, sel);
    const uint32_t lo = __byte_perm(t.l0, t.l1, sel);
    // the codes' sign bits in the top bits of four bytes
    hi |= __byte_perm(w, w4, half ? 0x3726 : 0x1504) & 0x80808080u;
    o[2 * half] = __byte_perm(lo, hi, 0x5140);
    o[2 * half + 1] = __byte_perm(lo, hi, 0x7362);
  }
}

// Partial scores of this warp: Q over dims 128kq..+128 and rope dims 16kq..+16 against
// keys 32kh..32kh+31 of the tile at raw.  c[j]: keys 32kh + 8j..+8.
__device__ __forceinline__ void kv4_qk(const uint8_t* raw, const uint32_t (&qa)[9][4], int kq,
                                       int kh, int lane, float (&c)[4][4]) {
  const int g = lane >> 2, cq = lane & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint8_t* row = raw + (32 * kh + 8 * j + g) * KV4_ROW_BYTES;
    const uint4 w = *reinterpret_cast<const uint4*>(row + 64 * kq + 16 * cq);
    const E2m1Table t = e2m1_table(row[256 + 4 * kq + cq]);
    c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.f;
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t o[4];
      e2m1_expand(ws[i], t, o);
      mma_bf16(c[j], qa[2 * i], o[0], o[1]);
      mma_bf16(c[j], qa[2 * i + 1], o[2], o[3]);
    }
  }
  const uint32_t rope = smem_u32(raw) + (32 * kh + (lane & 7) + 8 * (lane >> 4)) * KV4_ROW_BYTES +
                        272 + 32 * kq + 16 * ((lane >> 3) & 1);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t b0, b1, b2, b3;
    ldsm_x4(rope + 16 * j * KV4_ROW_BYTES, b0, b1, b2, b3);
    mma_bf16(c[2 * j], qa[8], b0, b1);
    mma_bf16(c[2 * j + 1], qa[8], b2, b3);
  }
}

// O = alpha O + P V over the tile at raw, for dims 64w..64w+63.  Output column n of MMA j
// is dim 64w + 8n + j.
__device__ __forceinline__ void kv4_pv(const uint8_t* raw, uint32_t pbase, float al0, float al1,
                                       int warp, int lane, float (&o)[8][4]) {
  const int g = lane >> 2, cq = lane & 3;
  const E2m1Table t{0x3F3F3F00u, 0x40404040u, 0xC0800000u, 0xC0804000u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    o[i][0] *= al0;
    o[i][1] *= al0;
    o[i][2] *= al1;
    o[i][3] *= al1;
  }
  const int pr = (lane & 7) + 8 * ((lane >> 3) & 1);
#pragma unroll
  for (int ks = 0; ks < K4_BK / 16; ++ks) {
    uint32_t pa[4];
    ldsm_x4(pbase + (pr * K4_PROW + 16 * ks + 8 * (lane >> 4)) * 2, pa[0], pa[1], pa[2], pa[3]);
    uint32_t v[2][8];  // [keys +0,1 / +8,9][dim]
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint8_t* ra = raw + (16 * ks + 8 * hf + 2 * cq) * KV4_ROW_BYTES;
      const uint8_t* rb = ra + KV4_ROW_BYTES;
      const uint32_t wa = *reinterpret_cast<const uint32_t*>(ra + 32 * warp + 4 * g);
      const uint32_t wb = *reinterpret_cast<const uint32_t*>(rb + 32 * warp + 4 * g);
      const uint32_t ea = ra[256 + 2 * warp + (g >> 2)], eb = rb[256 + 2 * warp + (g >> 2)];
      const uint32_t s = (ea << 7) | (eb << 23);
      // codes of both keys side by side: dims 0, 2, 4, 6 and 1, 3, 5, 7
      const uint32_t t0 = (wa & 0x0F0F0F0Fu) | ((wb << 4) & 0xF0F0F0F0u);
      const uint32_t t1 = ((wa >> 4) & 0x0F0F0F0Fu) | (wb & 0xF0F0F0F0u);
      uint32_t e0[4], e1[4];
      e2m1_expand(t0, t, e0);
      e2m1_expand(t1, t, e1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[hf][2 * i] = bf16x2_mul(e0[i], s);
        v[hf][2 * i + 1] = bf16x2_mul(e1[i], s);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) mma_bf16(o[j], pa, v[0][j], v[1][j]);
  }
}

__device__ __forceinline__ void kv4_consumer(Kv4Smem& sm, const AttnArgs& a) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &sm.abort;
  const int kq = warp >> 1, kh = warp & 1;  // QK: dim quarter, key half of the tile
  const int g = lane >> 2, cq = lane & 3;
  const int sh = 2 * warp + (lane >> 4);    // softmax: head of this lane
  const int sk = 4 * (lane & 15);           // and its four keys
  int stage = 0;
  uint32_t ph = 0;
  int rel = -1;  // stage of the previous tile, released after the next partial barrier
  const long nj = attn_nitems(a);
  auto store_partial = [&](const float (&c)[4][4]) {
    float* sp = &sm.s_part[kq][0][0] + 32 * kh + 2 * cq;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      *reinterpret_cast<float2*>(sp + g * K4_SROW + 8 * j) = make_float2(c[j][0], c[j][1]);
      *reinterpret_cast<float2*>(sp + (g + 8) * K4_SROW + 8 * j) = make_float2(c[j][2], c[j][3]);
    }
  };
  auto masks = [&](int st) { return *reinterpret_cast<const uint64_t*>(&sm.vmask[st][0]); };
  for (long it = 0; it < nj; ++it) {
    const AttnItem x = attn_item<K4_BK>(a, it);
    if (!mbar_wait(smem_u32(&sm.qfull), it & 1, abort, kErrTimeoutEpilogue)) return;
    uint32_t qa[9][4];
    {
      // dims 128kq + 32cq + 4i..+4 of heads g, g + 8: the order in which kv4_qk expands
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int ofs = (128 * kq + 32 * cq + 4 * i) * 2;
        const uint2 u = *reinterpret_cast<const uint2*>(&sm.q[g][ofs]);
        const uint2 v = *reinterpret_cast<const uint2*>(&sm.q[g + 8][ofs]);
        qa[i][0] = u.x;
        qa[i][1] = v.x;
        qa[i][2] = u.y;
        qa[i][3] = v.y;
      }
      ldsm_x4(smem_u32(&sm.q[(lane & 7) + 8 * ((lane >> 3) & 1)][0]) +
                  (AT_DV + 16 * kq + 8 * (lane >> 4)) * 2,
              qa[8][0], qa[8][1], qa[8][2], qa[8][3]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.qempty));
    float o[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m_run = -INFINITY, l_run = 0.f;  // softmax state of head sh (its 16 lanes agree)

    if (!mbar_wait(smem_u32(&sm.full[stage]), ph, abort, kErrTimeoutEpilogue)) return;
    int cur = stage, cur_last = sm.last[stage];
    uint64_t cur_vm = masks(stage);
    {
      float c[4][4];
      kv4_qk(&sm.raw[stage][0][0], qa, kq, kh, lane, c);
      store_partial(c);
    }
    if (++stage == K4_STAGES) {
      stage = 0;
      ph ^= 1;
    }
    for (;;) {
      named_bar_sync(1, AT_CONSUMERS);  // partials of cur complete, P V of prev done
      if (tid == 0 && rel >= 0) mbar_arrive(smem_u32(&sm.empty[rel]));
      const bool more = !cur_last;
      float c[4][4];
      int nxt = -1, nxt_last = 1;
      uint64_t nxt_vm = 0;
      if (more) {  // the next tile's QK runs under this tile's softmax
        if (!mbar_wait(smem_u32(&sm.full[stage]), ph, abort, kErrTimeoutEpilogue)) return;
        nxt = stage;
        nxt_last = sm.last[stage];
        nxt_vm = masks(stage);
        kv4_qk(&sm.raw[stage][0][0], qa, kq, kh, lane, c);
        if (++stage == K4_STAGES) {
          stage = 0;
          ph ^= 1;
        }
      }
      {
        float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) {
          const float4 u = *reinterpret_cast<const float4*>(&sm.s_part[qq][sh][sk]);
          z.x += u.x;
          z.y += u.y;
          z.z += u.z;
          z.w += u.w;
        }
        const unsigned vb = static_cast<unsigned>(cur_vm >> sk);
        z.x = (vb & 1u) ? z.x * a.scale_log2 : -INFINITY;
        z.y = (vb & 2u) ? z.y * a.scale_log2 : -INFINITY;
        z.z = (vb & 4u) ? z.z * a.scale_log2 : -INFINITY;
        z.w = (vb & 8u) ? z.w * a.scale_log2 : -INFINITY;
        float t = fmaxf(fmaxf(z.x, z.y), fmaxf(z.z, z.w));
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
        const float n = fmaxf(m_run, t);
        const float al = (n == -INFINITY) ? 1.f : fast_exp2(m_run - n);
        const float bse = (n == -INFINITY) ? 0.f : n;
        const float e0 = fast_exp2(z.x - bse), e1 = fast_exp2(z.y - bse);
        const float e2 = fast_exp2(z.z - bse), e3 = fast_exp2(z.w - bse);
        float rs = (e0 + e1) + (e2 + e3);
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) rs += __shfl_xor_sync(0xffffffffu, rs, off);
        l_run = l_run * al + rs;
        m_run = n;
        *reinterpret_cast<uint2*>(&sm.p[sh][sk]) = make_uint2(pack_bf16(e0, e1), pack_bf16(e2, e3));
        if ((lane & 15) == 0) sm.alpha[sh] = al;
      }
      named_bar_sync(1, AT_CONSUMERS);  // P, alpha complete
      kv4_pv(&sm.raw[cur][0][0], smem_u32(&sm.p[0][0]), sm.alpha[g], sm.alpha[g + 8], warp, lane, o);
      rel = cur;
      if (!more) break;
      store_partial(c);
      cur = nxt;
      cur_last = nxt_last;
      cur_vm = nxt_vm;
    }

    // ---- item epilogue: head h's final max and sum live in warp h/2
    named_bar_sync(1, AT_CONSUMERS);  // every warp's P V of the item is done
    if ((lane & 15) == 0) {
      sm.fin_m[sh] = m_run;
      sm.fin_l[sh] = l_run;
    }
    named_bar_sync(1, AT_CONSUMERS);
    // this lane holds dims 64 warp + 16cq..+16 of heads g (o[.][0..1]) and g + 8 (o[.][2..3])
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int h = g + 8 * hh;
      const float M = sm.fin_m[h], L = sm.fin_l[h];
      const int d = 64 * warp + 16 * cq;
      if (!a.split) {
        const float inv = L > 0.f ? 1.f / L : 0.f;
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // dims 2i, 2i + 1 of the 16
          const int j = 2 * (i & 3), n = 2 * hh + (i >> 2);
          u[i] = pack_bf16(o[j][n] * inv, o[j + 1][n] * inv);
        }
        uint32_t* ob = reinterpret_cast<uint32_t*>(a.out + (x.qrow * AT_H + h) * AT_DV + d);
        if ((reinterpret_cast<uintptr_t>(a.out) & 15) == 0) {
          reinterpret_cast<uint4*>(ob)[0] = make_uint4(u[0], u[1], u[2], u[3]);
          reinterpret_cast<uint4*>(ob)[1] = make_uint4(u[4], u[5], u[6], u[7]);
        } else {  // only required to be aligned to 4
#pragma unroll
          for (int i = 0; i < 8; ++i) ob[i] = u[i];
        }
        if (a.lse && warp == 0 && cq == 0)
          a.lse[x.qrow * AT_H + h] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
      } else {
        float* po = a.part_o + (x.pslot * AT_H + h) * AT_DV + d;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // dims 4i..4i+3
          const int j = 4 * (i & 1), n = 2 * hh + (i >> 1);
          *reinterpret_cast<float4*>(po + 4 * i) =
              make_float4(o[j][n], o[j + 1][n], o[j + 2][n], o[j + 3][n]);
        }
        if (warp == 0 && cq == 0) {
          a.part_ml[(x.pslot * AT_H + h) * 2] = M;
          a.part_ml[(x.pslot * AT_H + h) * 2 + 1] = L;
        }
      }
    }
  }
}

__global__ void __launch_bounds__(K4_THREADS, 1)
    attn_kv4_kernel(const AttnArgs a, const __grid_constant__ PagedArgs pg) {
  extern __shared__ uint8_t at_smem_raw[];
  Kv4Smem& sm = *reinterpret_cast<Kv4Smem*>(
      (reinterpret_cast<uintptr_t>(at_smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  if (threadIdx.x == 0) {
    for (int s = 0; s < K4_STAGES; ++s) {
      // every producer thread's copies, and one arrival per warp after its flags
      mbar_init(smem_u32(&sm.full[s]), 32 * K4_PROD_WARPS + K4_PROD_WARPS);
      mbar_init(smem_u32(&sm.empty[s]), 1);
    }
    mbar_init(smem_u32(&sm.qfull), 1);
    mbar_init(smem_u32(&sm.qempty), AT_CONSUMERS / 32);
    mbar_init(smem_u32(&sm.ifull[0]), 1);
    mbar_init(smem_u32(&sm.ifull[1]), 1);
    mbar_init(smem_u32(&sm.pitem), K4_PROD_WARPS);
    sm.abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  grid_dep_wait();  // set-up above touches no global memory
  if (threadIdx.x >= AT_CONSUMERS)
    kv4_producer(sm, a, pg);
  else
    kv4_consumer(sm, a);
  __syncthreads();
}

static ic_status launch_attn_kv4(const AttnArgs& a, const PagedArgs& pg, long grid,
                                 cudaStream_t stream) {
  const int smem = static_cast<int>(sizeof(Kv4Smem)) + 128;
  ic_status st = cuda_check(cudaFuncSetAttribute(attn_kv4_kernel,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                            "cudaFuncSetAttribute(attn_kv4)");
  if (st) return st;
  return cuda_check(launch_dep(attn_kv4_kernel, dim3(static_cast<unsigned>(grid)),
                               dim3(K4_THREADS), smem, stream, 1, a, pg),
                    "attn_kv4_kernel launch");
}
