// attention.cu -- decode attention over the whole cache: the kernel over the
// packed tiles (attention.cuh) and the tail, and the probe of its bounded
// waits.
#include "attention.cuh"

namespace kivi {
namespace {

// The slot the epoch probe waits on: it stays 0, and the probe waits for 1.
__device__ unsigned g_probe_epoch;

// Diagnostics: one thread waits, with the bounded wait of the staged tiles, on
// phase 0 of an mbarrier that nothing completes (no copy is issued, no thread
// arrives), and records the timeout in *status as a packed split does in the
// workspace status word; then the same for the epoch wait.
__global__ void wait_probe_kernel(int* status) {
  __shared__ __align__(8) unsigned long long bar;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    mbar_fence_init();
    if (!mbar_wait(&bar, 0u)) atomicOr(status, 1);
    if (!epoch_wait(&g_probe_epoch, 1u)) atomicOr(status, 2);
  }
}

// ---------------------------------------------------------------------------
// A tail split on CUDA cores: tokens [c0, c0 + n), n <= kTailTok, of the tail
// [t_tail, l), staged in one round of copies (fp16 residual rows, packed rows
// and the key groups' scales / zeros), for the chunk's 4 NQ query heads.
// Scores: warp w takes tokens w, w + 4, ..., lane l channels 4l .. 4l + 3,
// and one transposing butterfly over the lanes sums the 4 NQ heads at once;
// the softmax of a head is one warp; values take one thread per channel.
// Keys and values of packed rows are dequantized as c * s + z with a single
// rounding, which equals the notebook's fl(fl(c * s) + z) because c * s is
// exact in fp32.  Leaves the partial of the CTA in warp 0's slots (the other
// warps' slots empty) and its output rows in `mo0` ([kNH][kHeadDim], inside
// the staged key rows).

// Sum of v[0..H) over the 32 lanes, H heads at once: each butterfly level
// halves the values a lane carries (the lanes with bit `o` set keep the upper
// half), then plain levels finish the sums.  Every lane of a block of 32 / H
// lanes ends with the total of head `head`.
template <int H>
__device__ __forceinline__ float reduce_heads(const float (&v)[H], int lane, int& head) {
  float cur[H];
#pragma unroll
  for (int i = 0; i < H; ++i) cur[i] = v[i];
  head = 0;
  int o = 16;
#pragma unroll
  for (int half = H / 2; half >= 1; half >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = up ? cur[i + half] : cur[i];
      const float send = up ? cur[i] : cur[i + half];
      cur[i] = keep + __shfl_xor_sync(kFull, send, o);
    }
    head += up ? half : 0;
    o >>= 1;
  }
#pragma unroll
  for (; o > 0; o >>= 1) cur[0] += __shfl_xor_sync(kFull, cur[0], o);
  return cur[0];
}

template <int BITS, int NQ>
__device__ __noinline__ void tail_split(const CacheView& cv, const AttnArgs& a, const SeqPlan p, TailSmem<BITS>& ts,
                                        float* mo0, long unit, int b, int j0, int nh, int c0, uint32_t round,
                                        float (&s_m)[kWarps][kNH], float (&s_l)[kWarps][kNH]) {
  constexpr int L = (1 << BITS) - 1;
  constexpr int RB = kHeadDim * BITS / 8;  // packed row bytes
  constexpr int H = 4 * NQ;                // heads of this tail
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = min(kTailTok, p.l - c0);
  const int nk = max(0, min(n, p.nq_k - c0));  // rows [0, nk) hold packed keys
  const int nv = max(0, min(n, p.nq_v - c0));  // rows [0, nv) hold packed values
  const int ngk = (nk + kGroup - 1) / kGroup, ngv = (nv + kGroup - 1) / kGroup;
  const int tile0 = c0 / kGroup;  // c0 is a multiple of 32: packed rows span at most two tiles

  // ---- stage the round with bulk copies (thread 0), and q ----
  if (tid == 0) {
    if (round == 0) {
      mbar_init(&ts.bar, 1);
      mbar_fence_init();
    }
    fence_proxy_async();  // the buffers were last used by ordinary loads and stores
    const int ob = outlier_block_bytes(cv.n_out);
    const int wk = n - nk, wv = n - nv;  // residual rows of keys / values
    const int sk0 = (int)((c0 + nk) % cv.W), sv0 = (int)((c0 + nv) % cv.W);
    const int k1 = min(wk, cv.W - sk0), v1 = min(wv, cv.W - sv0);  // first runs of ring slots
    const uint32_t bytes = (uint32_t)(ngk * (kGroup * RB + 4 * kHeadDim + ob) + ngv * (kGroup * RB + 4 * kHeadDim) +
                                      (wk + wv) * 2 * kHeadDim);
    mbar_expect_tx(&ts.bar, bytes);
    for (int gi = 0; gi < ngk; ++gi) {
      const uint8_t* tile = tile_at<BITS>(cv, unit, tile0 + gi);
      bulk_g2s(ts.kpk[gi], tile + kOffKc<BITS>, kGroup * RB, &ts.bar);
      bulk_g2s(ts.kg[gi][0], tile + kOffSk<BITS>, 2 * kHeadDim, &ts.bar);  // scales
      bulk_g2s(ts.kg[gi][1], tile + kOffZk, 2 * kHeadDim, &ts.bar);        // zeros
      if (ob) bulk_g2s(ts.ko[gi], tile + kTileBytes<BITS>, ob, &ts.bar);
    }
    for (int gi = 0; gi < ngv; ++gi) {
      const uint8_t* tile = tile_at<BITS>(cv, unit, tile0 + gi);
      bulk_g2s(ts.vpk[gi], tile + kOffVc<BITS>, kGroup * RB, &ts.bar);
      bulk_g2s(ts.vg[gi], tile + kOffSv<BITS>, 4 * kHeadDim, &ts.bar);
    }
    const __half* rk = cv.ring_k + unit * cv.W * kHeadDim;
    const __half* rv = cv.ring_v + unit * cv.W * kHeadDim;
    if (k1 > 0) bulk_g2s(ts.kring[nk], rk + (long)sk0 * kHeadDim, k1 * 2 * kHeadDim, &ts.bar);
    if (wk > k1) bulk_g2s(ts.kring[nk + k1], rk, (wk - k1) * 2 * kHeadDim, &ts.bar);
    if (v1 > 0) bulk_g2s(ts.vring[nv], rv + (long)sv0 * kHeadDim, v1 * 2 * kHeadDim, &ts.bar);
    if (wv > v1) bulk_g2s(ts.vring[nv + v1], rv, (wv - v1) * 2 * kHeadDim, &ts.bar);
  }
  {
    float qj[kNH];
#pragma unroll
    for (int j = 0; j < kNH; ++j)
      qj[j] = j < nh ? load_q(a.q, ((long)b * a.Hq + j0 + j) * kHeadDim + tid, a.q_dtype) * a.scale_log2 : 0.0f;
    ts.q8[tid][0] = make_float4(qj[0], qj[1], qj[2], qj[3]);
    ts.q8[tid][1] = make_float4(qj[4], qj[5], qj[6], qj[7]);
  }
  __syncthreads();  // q staged; the barrier initialized before anyone waits on it
  if (!mbar_wait(&ts.bar, round & 1u) && tid == 0) atomicOr(a.status, 1);

  // ---- scores: warp w takes tokens w, w + 4, ... (two at a time); lane l
  //      channels 4l..4l+3 ----
  {
    float qr[4][H];  // q of this lane's channels, the tail's heads
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) {
        const float4 v = ts.q8[4 * lane + c][nq];
        qr[c][4 * nq] = v.x;
        qr[c][4 * nq + 1] = v.y;
        qr[c][4 * nq + 2] = v.z;
        qr[c][4 * nq + 3] = v.w;
      }
    // scales / zeros of this lane's channels in the (at most two) key groups
    float ks_[2][4], kz_[2][4];
#pragma unroll
    for (int gi = 0; gi < 2; ++gi)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int pos = kscale_pos<BITS>(4 * lane + c);
        ks_[gi][c] = gi < ngk ? __half2float(reinterpret_cast<const __half*>(ts.kg[gi][0])[pos]) : 0.0f;
        kz_[gi][c] = gi < ngk ? __half2float(reinterpret_cast<const __half*>(ts.kg[gi][1])[pos]) : 0.0f;
      }
    auto score = [&](int r, float (&acc)[H]) {
      float kx[4];
      if (r < nk) {
        uint32_t cd[4];
        key_codes4<BITS>(ts.kpk[r >> 5] + (r & 31) * RB, r & 31, lane, cd);
        const int gi = r >> 5;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          kx[c] = fmaf(__uint_as_float(cd[c] | 0x4B000000u) - 8388608.0f, gi ? ks_[1][c] : ks_[0][c],
                       gi ? kz_[1][c] : kz_[0][c]);
      } else {
        const uint2 h4 = *reinterpret_cast<const uint2*>(&ts.kring[r][4 * lane]);
        kx[0] = h_lo(h4.x);
        kx[1] = h_hi(h4.x);
        kx[2] = h_lo(h4.y);
        kx[3] = h_hi(h4.y);
      }
#pragma unroll
      for (int j = 0; j < H; ++j) {
        acc[j] = kx[0] * qr[0][j];
#pragma unroll
        for (int c = 1; c < 4; ++c) acc[j] = fmaf(kx[c], qr[c][j], acc[j]);
      }
      if (lane == 0 && r < nk && cv.n_out > 0) {
        // the group's fp16 outlier channels (their packed codes decode to 0)
        const uint32_t iw = ts.ko[r >> 5][0];
        const __half* ov = reinterpret_cast<const __half*>(&ts.ko[r >> 5][4]);
        for (int o = 0; o < cv.n_out; ++o) {
          const float x = __half2float(ov[(r & 31) * cv.n_out + o]);
          const float* qo = reinterpret_cast<const float*>(&ts.q8[(iw >> (8 * o)) & 0xffu][0]);
#pragma unroll
          for (int j = 0; j < H; ++j) acc[j] = fmaf(x, qo[j], acc[j]);
        }
      }
    };
#pragma unroll 1
    for (int r = warp; r < n; r += 2 * kWarps) {
      const int r1 = r + kWarps < n ? r + kWarps : r;  // a second token (or the first again)
      float acc0[H], acc1[H];
      score(r, acc0);
      score(r1, acc1);
      int head;
      const float s0 = reduce_heads<H>(acc0, lane, head);
      const float s1 = reduce_heads<H>(acc1, lane, head);
      if ((lane & (32 / H - 1)) == 0) {
        reinterpret_cast<float*>(ts.p8)[r * kNH + head] = s0;
        reinterpret_cast<float*>(ts.p8)[r1 * kNH + head] = s1;
      }
    }
  }
  __syncthreads();

  // ---- softmax of heads `warp` (and `warp` + 4) over the round ----
#pragma unroll
  for (int hh = 0; hh < NQ; ++hh) {
    const int j = warp + kWarps * hh;
    float* pj = reinterpret_cast<float*>(ts.p8) + j;  // [token][kNH]
    const float x0 = lane < n ? pj[kNH * lane] : -INFINITY;
    const float x1 = lane + 32 < n ? pj[kNH * (lane + 32)] : -INFINITY;
    const float mx = warp_max(fmaxf(x0, x1));
    const float e0 = lane < n ? fast_exp2(x0 - mx) : 0.0f;
    const float e1 = lane + 32 < n ? fast_exp2(x1 - mx) : 0.0f;
    pj[kNH * lane] = e0;
    pj[kNH * (lane + 32)] = e1;
    const float sum = warp_sum(e0 + e1);
    if (lane == 0) {
      ts.mh[j] = mx;
      ts.lh[j] = sum;
    }
  }
  __syncthreads();

  // ---- values: thread d accumulates channel d of the tail's heads ----
  const int d = tid;
  const int vpos = v_unit_pos(d >> 2);
  const int vsh = BITS * (d & 3);
  float o[H];
#pragma unroll
  for (int j = 0; j < H; ++j) o[j] = 0.0f;
#pragma unroll 2
  for (int r = 0; r < n; ++r) {
    float vx;
    if (r < nv) {
      const uint8_t* row = ts.vpk[r >> 5] + (r & 31) * RB;
      uint32_t cb;
      if constexpr (BITS == 2) cb = row[vpos];
      else if constexpr (BITS == 3) cb = row[vpos] | ((uint32_t)*reinterpret_cast<const uint16_t*>(row + kHiPlane3 + 2 * ((d & 31) >> 2)) << 8);
      else if constexpr (BITS == 4) cb = *reinterpret_cast<const uint16_t*>(row + 2 * vpos);
      else cb = *reinterpret_cast<const uint32_t*>(row + vrow_byte<8>(r & 31, 4 * vpos));
      const int vs = vscale_pos(r & 31, d >> 5);
      const float sv = __half2float(reinterpret_cast<const __half*>(ts.vg[r >> 5][0])[vs]);
      const float zv = __half2float(reinterpret_cast<const __half*>(ts.vg[r >> 5][1])[vs]);
      float cf;
      if constexpr (BITS == 3) {
        // low two bits from the unit's byte, the high bit from bits 8.. (the high unit)
        const uint32_t lo = (cb >> (2 * (d & 3))) & 3u;
        const uint32_t hi = (cb >> (8 + hi_bit3(d >> 6, 4 * ((d >> 5) & 1) + (d & 3)))) & 1u;
        cf = (float)(lo | (hi << 2));
      } else {
        cf = __uint_as_float(((cb >> vsh) & L) | 0x4B000000u) - 8388608.0f;
      }
      vx = fmaf(cf, sv, zv);
    } else {
      vx = __half2float(ts.vring[r][d]);
    }
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      const float4 pr = ts.p8[r][nq];
      o[4 * nq] = fmaf(pr.x, vx, o[4 * nq]);
      o[4 * nq + 1] = fmaf(pr.y, vx, o[4 * nq + 1]);
      o[4 * nq + 2] = fmaf(pr.z, vx, o[4 * nq + 2]);
      o[4 * nq + 3] = fmaf(pr.w, vx, o[4 * nq + 3]);
    }
  }
  __syncthreads();  // every thread is done with the staged rows (the merge area)

#pragma unroll
  for (int j = 0; j < H; ++j) mo0[j * kHeadDim + d] = o[j];
  if (lane < kNH) {
    s_m[warp][lane] = warp == 0 && lane < H ? ts.mh[lane] : -INFINITY;
    s_l[warp][lane] = warp == 0 && lane < H ? ts.lh[lane] : 0.0f;
  }
}

// Packed tiles [tile0, tile1) of one (batch, kv-head, head chunk) on the
// tensor cores.  Warp w takes tiles tile0 + w, + kWarps, ... through its own
// ring of staged tiles (lane 0 issues the copies; no CTA barrier in the
// loop).  Leaves each warp's (max, sum) per head in s_m / s_l and its output
// in its merge area.
template <int BITS, int NB>
__device__ void packed_split(const CacheView& cv, const AttnArgs& a, const SmemView<BITS, NB>& sv, long unit, int b,
                             int j0, int nh, int tile0, int tile1, float (&s_m)[kWarps][kNH],
                             float (&s_l)[kWarps][kNH]) {
  const int kStages = sv.S;
  PackedState<NB>& ws = sv.ps();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tig = lane & 3;
  const int n_mine = tile0 + warp < tile1 ? (tile1 - tile0 - warp + kWarps - 1) / kWarps : 0;
  unsigned char* const ring = reinterpret_cast<unsigned char*>(sv.ring(warp));
  auto st = [&](int k) -> TileBuf<BITS>& { return *reinterpret_cast<TileBuf<BITS>*>(ring + (size_t)k * sv.stride); };
  unsigned long long* bars = ws.bar[warp];
  const float* const qo = sv.qo();  // q for the outlier channels (when the cache keeps them)
  float qv8[8];
  load_q8(a, b, j0, nh, qv8);

  if (lane == 0) {
    for (int k = 0; k < kStages; ++k) mbar_init(&bars[k], 1);
    mbar_fence_init();
  }
  __syncwarp();
  const UnitSrc us = unit_src<BITS>(cv, a, unit, 0);
  const int t_first = tile0 + warp;  // this warp's tiles: t_first + kWarps * k
  int issued = min(n_mine, kStages);
  // the first tile before the q tables, the other stages after them: at
  // launch every warp of the GPU issues at once, and the first tile (and the
  // tables) should not queue behind the later stages.  A dependent launch
  // whose packed tiles the append may write builds the tables while the
  // append runs and issues every copy after it.
  const bool wait_first = a.pdl == kPdlAll;
  if (!wait_first && lane == 0 && issued > 0) issue_tile<BITS>(st(0), &bars[0], us, t_first);
  // the key zeros of the first sixteen tiles are loaded before the tables
  // are built (unless the tiles may still be written by the kernel before)
  uint4 z[2][4];
  if (!wait_first) load_zk<BITS>(us, t_first, n_mine, 0, g, tig, z);
  build_q_tables<BITS, NB>(sv, a, qv8, cv.n_out > 0);
  __syncthreads();
  if (wait_first) grid_dependency_wait();
  if (lane == 0)
    for (int k = wait_first ? 0 : 1; k < issued; ++k) issue_tile<BITS>(st(k), &bars[k], us, t_first + kWarps * k);
  float* const brows = &ws.beta[warp][0][0];
  if (n_mine > 0) {
    if (wait_first) load_zk<BITS>(us, t_first, n_mine, 0, g, tig, z);
    beta_mma<NB>(ws, z, g, tig, brows);
    if (n_mine > 16) {
      load_zk<BITS>(us, t_first, n_mine, 16, g, tig, z);
      beta_mma<NB>(ws, z, g, tig, brows + 16 * 4 * NB);
    }
    __syncwarp();
  }
  float ks[NB], m_run[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    ks[nb] = ws.qscale[NB == 1 ? tig : 2 * tig + nb];
    m_run[nb] = -INFINITY;
  }

  float O[8][4], Z[4];
#pragma unroll
  for (int mt = 0; mt < 8; ++mt)
#pragma unroll
    for (int i = 0; i < 4; ++i) O[mt][i] = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) Z[i] = 0.0f;

  // Tile k's scores are computed one iteration ahead of its values: the
  // scores of tile k + 1 and the values of tile k form one straight-line
  // block (the wait for tile k + 1 comes first), so that their independent
  // MMA chains can interleave.  One loop body walks the ring with the stage
  // as a run-time index.
  int done = 0;
  bool failed = false;
  uint32_t pb[2][2];  // the staged tile's weights as value B fragments
  uint32_t pl[2][2];  // (unused: see softmax_p)
  float ts[NB];
  if (n_mine > 0) {
    bool ok = mbar_try_wait(&bars[0], 0u);
    if (!ok) ok = mbar_wait(&bars[0], 0u);
    if (__any_sync(kFull, !ok)) {
      failed = true;
    } else {
      float sc[NB][4], mb[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mb[nb] = 0.0f;
      key_scores<BITS, NB>(ws, st(0), g, tig, ks, mb, cv.n_out, qo, brows, sc);
      softmax_p<BITS, NB, kAttnAll>(sc, g, tig, m_run, O, Z, pb, pl, ts);
    }
  }
  int k = 0, sk = 0;     // tile whose values are next, and its stage
  uint32_t parn = 0;     // phase parity of the stage of tile k + 1
  // source of the next tile to stage (tile k + kStages of this warp)
  const long src_step = (long)kWarps * us.stride;
  const uint8_t* next_src = us.tiles + (long)(t_first + kWarps * kStages) * us.stride + kStageOff;
  while (!failed && k + 1 < n_mine) {
    const int sn = sk + 1 == kStages ? 0 : sk + 1;  // stage of tile k + 1
    if (sn == 0) parn ^= 1u;
    if (!__all_sync(kFull, mbar_try_wait(&bars[sn], parn))) {
      const bool ok = mbar_wait(&bars[sn], parn);
      if (__any_sync(kFull, !ok)) {
        failed = true;
        break;
      }
    }
    const int kb = (k + 1) % kBetaTiles;  // beta row of tile k + 1
    if (kb == 0) {
      // the next block of kBetaTiles tiles (every row of the last one is read)
      __syncwarp();
      uint4 zz[2][4];
      load_zk<BITS>(us, t_first, n_mine, k + 1, g, tig, zz);
      beta_mma<NB>(ws, zz, g, tig, brows);
      if (k + 17 < n_mine) {
        load_zk<BITS>(us, t_first, n_mine, k + 17, g, tig, zz);
        beta_mma<NB>(ws, zz, g, tig, brows + 16 * 4 * NB);
      }
      __syncwarp();
    }
    float sc[NB][4];
    key_scores<BITS, NB>(ws, st(sn), g, tig, ks, m_run, cv.n_out, qo, brows + kb * 4 * NB, sc);
    value_acc<BITS, NB, kAttnAll>(st(sk), pb, pl, g, tig, O, Z);
    done = k + 1;
    __syncwarp();  // every lane is done with stage sk
    const bool more = k + kStages < n_mine;
    issue_tile_if<BITS>(more && lane == 0, st(sk), &bars[sk], next_src, us.copy);
    next_src += src_step;
    issued += more;
    softmax_p<BITS, NB, kAttnAll>(sc, g, tig, m_run, O, Z, pb, pl, ts);
    ++k;
    sk = sn;
  }
  if (!failed && n_mine > 0) {
    value_acc<BITS, NB, kAttnAll>(st(sk), pb, pl, g, tig, O, Z);  // the last tile's values
    done = n_mine;
  }
  if (done < n_mine) {
    // A wait timed out: record it, and let every copy still in flight land
    // before the warp's buffers are reused (each wait bounded again).
    if (lane == 0) atomicOr(a.status, 1);
    for (int kk = done; kk < issued; ++kk) mbar_wait(&bars[kk % kStages], (uint32_t)((kk / kStages) & 1));
    __syncwarp();
  } else if (lane == 0) {
    // every copy has landed: the barriers' memory may be reused
    for (int kk = 0; kk < kStages; ++kk) mbar_inval(&bars[kk]);
  }

  // ---- this warp's partial: max, sum and output per head ----
  // The value columns of lane (g, tig) are heads 2 tig and 2 tig + 1: their
  // weight sums are Z[2], Z[3] (the all-ones rows); the running max of head
  // hd(nb) of key_scores is m_run[nb] of the lanes with this tig.
  if (g == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (NB == 2) s_m[warp][2 * tig + i] = n_mine > 0 ? m_run[i] : -INFINITY;
      else s_m[warp][4 * i + tig] = i == 0 && n_mine > 0 ? m_run[0] : -INFINITY;
    }
    s_l[warp][2 * tig] = Z[2];
    s_l[warp][2 * tig + 1] = Z[3];
  }
  // z-term of value group gp for heads (2 tig, 2 tig + 1): Z[0], Z[1] of lane (gp, tig)
  float zt[4][2];
#pragma unroll
  for (int gp = 0; gp < 4; ++gp) {
    zt[gp][0] = __shfl_sync(kFull, Z[0], 4 * gp + tig);
    zt[gp][1] = __shfl_sync(kFull, Z[1], 4 * gp + tig);
  }
  if (n_mine == 0) return;  // no tile: the area stays unwritten (max -inf)
  float* oa = sv.merge_area(warp, kPathMma) + (2 * tig) * kHeadDim;
  float* ob = oa + kHeadDim;
#pragma unroll
  for (int mt = 0; mt < 8; ++mt) {
    const int gp = mt >> 1, hm = mt & 1;
    // code positions of rows g and g + 8 of m-tile mt
    const int i_lo = BITS <= 3 ? 4 * (gp & 1) + 2 * hm : 2 * hm;
    const int ch = 32 * gp + 4 * g + 2 * hm;
    const float f_lo = kTwo24 * code_scale<BITS>(i_lo);
    const float f_hi = kTwo24 * code_scale<BITS>(i_lo + 1);
    oa[ch] = O[mt][0] * f_lo + zt[gp][0];
    ob[ch] = O[mt][1] * f_lo + zt[gp][1];
    oa[ch + 1] = O[mt][2] * f_hi + zt[gp][0];
    ob[ch + 1] = O[mt][3] * f_hi + zt[gp][1];
  }
}

// The tail on the last packed split (when no tail split fits the budget):
// the warps' packed partials are merged into registers, the tail rounds run
// one after another and are folded in, and the result is left as warp 0's
// slot (the other warps' slots empty) for the CTA merge.
template <int BITS, int NB>
__device__ void fused_tail(const CacheView& cv, const AttnArgs& a, const SeqPlan p, const SmemView<BITS, NB>& sv,
                           long unit, int b, int j0, int nh, float (&s_m)[kWarps][kNH],
                           float (&s_l)[kWarps][kNH]) {
  const int d = threadIdx.x;
  float pm[kNH], pl[kNH], po[kNH];
#pragma unroll
  for (int j = 0; j < kNH; ++j) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][j]);
    float lt = 0.0f, ot = 0.0f;
    if (M != -INFINITY) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (s_m[w][j] == -INFINITY) continue;
        const float e = fast_exp2(s_m[w][j] - M);
        lt += e * s_l[w][j];
        ot += e * sv.merge_area(w, kPathMma)[j * kHeadDim + d];
      }
    }
    pm[j] = M;
    pl[j] = lt;
    po[j] = ot;
  }
  __syncthreads();  // the warps' slots are read; the tail may overwrite them
  float* mo0 = sv.merge_area(0, kPathTail);
  uint32_t round = 0;
  for (int c0 = p.t_tail; c0 < p.l; c0 += kTailTok, ++round) {
    tail_split<BITS, NB>(cv, a, p, sv.tail(), mo0, unit, b, j0, nh, c0, round, s_m, s_l);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kNH; ++j) {
      const float tm = s_m[0][j];
      const float M = fmaxf(pm[j], tm);
      const float e1 = pm[j] == -INFINITY ? 0.0f : fast_exp2(pm[j] - M);
      const float e2 = tm == -INFINITY ? 0.0f : fast_exp2(tm - M);
      // (rows of heads the tail does not serve are not written: max -inf)
      po[j] = po[j] * e1 + (tm == -INFINITY ? 0.0f : mo0[j * kHeadDim + d] * e2);
      pl[j] = pl[j] * e1 + s_l[0][j] * e2;
      pm[j] = M;
    }
    __syncthreads();  // before the next round overwrites the staged rows
  }
  float* out0 = sv.merge_area(0, kPathMma);
#pragma unroll
  for (int j = 0; j < kNH; ++j) out0[j * kHeadDim + d] = po[j];
  if (d < kWarps * kNH) {
    const int w = d / kNH, j = d % kNH;
    float mj = pm[0], lj = pl[0];
#pragma unroll
    for (int i = 1; i < kNH; ++i) {
      mj = j == i ? pm[i] : mj;
      lj = j == i ? pl[i] : lj;
    }
    s_m[w][j] = w == 0 ? mj : -INFINITY;
    s_l[w][j] = w == 0 ? lj : 0.0f;
  }
  __syncthreads();
}

// grid (splits, H * head_chunks, B), 128 threads.
template <int BITS, int NB>
__global__ void __launch_bounds__(128, attn_ctas_per_sm(BITS, NB))
    attn_kernel(CacheView cv, AttnArgs a, const SeqLens lens) {
  extern __shared__ __align__(16) unsigned char smem_raw[];  // attn_stages: the tail or the packed layout
  const SmemView<BITS, NB> sv{smem_raw, a.stages, (uint32_t)(cv.tile_bytes - kStageOff)};
  __shared__ float s_m[kWarps][kNH], s_l[kWarps][kNH];
  __shared__ bool s_last;

  // Programmatic dependents of this launch (an overlapping attention call,
  // the next decode step's append) may start early.  An ordinary or an
  // overlapping launch lets them start at once: it writes nothing they read
  // (its workspace and out aside, which they wait for before writing), and
  // every kernel before it has completed or writes nothing it reads.  A
  // decode step's attention lets them start only once its append has
  // completed (before the merge below), so that no early start ever runs
  // ahead of a cache write.
  const bool step_launch = a.pdl == kPdlAll || a.pdl == kPdlTail;
  const int s = blockIdx.x;
  const int nhc = gridDim.y / cv.H;
  const int h = nhc == 1 ? (int)blockIdx.y : (int)blockIdx.y / nhc;
  const int hc = nhc == 1 ? 0 : (int)blockIdx.y % nhc;
  const int b = blockIdx.z;
  const long gid = (long)b * gridDim.y + blockIdx.y;  // (batch, kv-head, head chunk)
  // An overlapping launch releases its dependents at once, once its
  // generation ticket is taken (take_ticket); a decode step's attention
  // releases them once its append has completed (before the merge below),
  // an ordinary launch at its exit.
  const bool tickets = a.epoch_on && a.pdl != 0;
  unsigned gen = 0;  // thread 0: this launch's generation for the group
  if (tickets && threadIdx.x == 0) gen = take_ticket(a, gid);
  if (a.pdl == kPdlOverlap) {
    if (threadIdx.x == 0) gen = ticket_gen(gen);
    __syncthreads();
    grid_launch_dependents();
  }
  const int grp = a.Hq / cv.H;
  const int j0 = h * grp + hc * kNH;
  const int nh = min(kNH, grp - hc * kNH);
  const long unit = (long)b * cv.H + h;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  (void)gid;
  // this sequence's plan; splits past its own count have nothing to do (and
  // are not counted by its merge)
  const SeqPlan p = lens.uniform >= 0 ? a.plan : make_plan(lens.l[b], cv.R, cv.policy, a.scfg);
  if (s >= p.splits) {
    if (step_launch && threadIdx.x == 0) gen = ticket_gen(gen);  // the ticket is in before the exit
    return;
  }
  const int path = s < p.tail_splits ? kPathTail : kPathMma;

  if (path == kPathTail) {
    // the tail reads the rings the append writes
    if (a.pdl == kPdlAll || a.pdl == kPdlTail) grid_dependency_wait();
    tail_split<BITS, NB>(cv, a, p, sv.tail(), sv.merge_area(0, kPathTail), unit, b, j0, nh,
                         p.t_tail + s * kTailTok, 0u, s_m, s_l);
  } else {
    // ---- tensor cores: packed tiles [sp*chunk, min(t_tail, (sp+1)*chunk)) ----
    const int sp = s - p.tail_splits;
    const int tile0 = sp * p.chunk / 32;
    const int tile1 = min(p.t_tail, (sp + 1) * p.chunk) / 32;
    packed_split<BITS, NB>(cv, a, sv, unit, b, j0, nh, tile0, tile1, s_m, s_l);
  }
  __syncthreads();
  if (path == kPathMma && p.tail_fused && s == p.splits - 1) {
    if (a.pdl == kPdlTail) grid_dependency_wait();  // the tail reads what the append wrote
    fused_tail<BITS, NB>(cv, a, p, sv, unit, b, j0, nh, s_m, s_l);
  }
  // a decode step's attention releases its dependents once its append has
  // completed
  if (step_launch) {
    grid_dependency_wait();
    if (threadIdx.x == 0) gen = ticket_gen(gen);
    __syncthreads();
    grid_launch_dependents();
  }
  // an overlapping launch orders its first workspace write of the group after
  // the previous call on this workspace has finished with the group's slots
  // (see epoch_wait); a wait that gives up sets bit 2 of the status word
  if (a.pdl == kPdlOverlap && a.epoch_on) {
    if (threadIdx.x == 0 && !epoch_wait(a.epochs + 2 * gid + 1, gen)) atomicOr(a.status, 2);
    __syncthreads();
  }

  // ---- merge the warps of this CTA into one partial per head ----
  const int d = threadIdx.x;
  for (int j = 0; j < nh; ++j) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][j]);
    float lt = 0.0f, ot = 0.0f;
    if (M != -INFINITY) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (s_m[w][j] == -INFINITY) continue;  // an empty warp (its area is not written)
        const float e = fast_exp2(s_m[w][j] - M);
        lt += e * s_l[w][j];
        ot += e * sv.merge_area(w, path)[j * kHeadDim + d];
      }
    }
    const long pidx = (gid * a.scfg.max_splits + s) * kNH + j;
    a.ws_o[pidx * kHeadDim + d] = ot;
    if (d == 0) {
      a.ws_ml[pidx * 2] = M;
      a.ws_ml[pidx * 2 + 1] = lt;
    }
  }

  // ---- the last CTA of each group of kMergeGroup splits merges the group;
  //      with more than one group, the last group merges the group results ----
  const int n_grp = (p.splits + kMergeGroup - 1) / kMergeGroup;
  const int grp_i = s / kMergeGroup;
  const int g_lo = grp_i * kMergeGroup, g_n = min(kMergeGroup, p.splits - g_lo);
  __syncthreads();
  if (threadIdx.x == 0) {
    int* counter = a.counters + gid * a.merge_groups + grp_i;
    s_last = count_in(counter) == g_n - 1;
    if (s_last) *counter = 0;  // every other CTA of the group has counted in
  }
  __syncthreads();
  if (!s_last) return;
  // warp w merges heads w and w + kWarps
  float4 o4[2];
  float lsum_h[2], m_h[2];
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int j = warp + kWarps * hh;
    if (j < nh)
      merge_partials(a.ws_o + (gid * a.scfg.max_splits + g_lo) * kNH * kHeadDim, a.ws_ml + (gid * a.scfg.max_splits + g_lo) * kNH * 2,
                     g_n, j, o4[hh], m_h[hh], lsum_h[hh]);
  }
  if (n_grp > 1) {
    // a group result: write it, then count the group in
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int j = warp + kWarps * hh;
      if (j < nh) {
        const long pidx = (gid * a.merge_groups + grp_i) * kNH + j;
        *reinterpret_cast<float4*>(a.ws_o1 + pidx * kHeadDim + 4 * lane) = o4[hh];
        if (lane == 0) {
          a.ws_ml1[pidx * 2] = m_h[hh];
          a.ws_ml1[pidx * 2 + 1] = lsum_h[hh];
        }
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int* counter = a.counters2 + gid;
      s_last = count_in(counter) == n_grp - 1;
      if (s_last) *counter = 0;
    }
    __syncthreads();
    if (!s_last) return;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int j = warp + kWarps * hh;
      if (j < nh)
        merge_partials(a.ws_o1 + gid * a.merge_groups * kNH * kHeadDim, a.ws_ml1 + gid * a.merge_groups * kNH * 2,
                       n_grp, j, o4[hh], m_h[hh], lsum_h[hh]);
    }
  }
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int j = warp + kWarps * hh;
    if (j >= nh) continue;
    const float inv = 1.0f / lsum_h[hh];
    const float r[4] = {o4[hh].x * inv, o4[hh].y * inv, o4[hh].z * inv, o4[hh].w * inv};
    const long oi = ((long)b * a.Hq + j0 + j) * kHeadDim + 4 * lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (a.q_dtype == kF32) static_cast<float*>(a.out)[oi + i] = r[i];
      else if (a.q_dtype == kF16) static_cast<__half*>(a.out)[oi + i] = __float2half_rn(r[i]);
      else static_cast<__nv_bfloat16*>(a.out)[oi + i] = __float2bfloat16_rn(r[i]);
    }
  }
  // the group's slots are free for the next call on this workspace: every
  // thread's reads of them precede the barrier, the release orders them
  if (tickets) {
    __syncthreads();
    if (threadIdx.x == 0) st_release_u32(a.epochs + 2 * gid + 1, (gen + 1u) & kGenMask);
  }
  // An overlapping launch completes only after the launch before it: group
  // 0's final CTA waits for it last of all, so that whatever follows this
  // launch on the stream (a copy, a memset, a host read after a sync) also
  // follows every launch before it; the other CTAs exit at once.
  if (a.pdl == kPdlOverlap && gid == 0) grid_dependency_wait();
}

template <int BITS, int NB>
constexpr bool kTailFits =
    attn_ctas_per_sm(BITS, NB) * (sizeof(TailSmem<BITS>) + 1024 + 512) <= 228 * 1024;
static_assert(kTailFits<2, 1> && kTailFits<2, 2> && kTailFits<3, 1> && kTailFits<3, 2> && kTailFits<4, 1> &&
                  kTailFits<4, 2> && kTailFits<8, 1> && kTailFits<8, 2>,
              "the tail split's layout fits the CTAs of an SM");

template <int BITS, int NB>
cudaError_t launch_bits(const dim3& grid, const CacheView& cv, AttnArgs a, const SeqLens& lens,
                        cudaStream_t st) {
  size_t smem = 0, cap = 0;
  a.stages = attn_stages<BITS, NB>((uint32_t)(cv.tile_bytes - kStageOff), cv.n_out, &smem);
  // The shared-memory opt-in is a per-device function attribute: set to the
  // largest size any outlier count asks for (the same on every call, so
  // that calls from several host threads cannot shrink it under another's
  // launch); setting it costs a host call only.
  const uint32_t plain = (uint32_t)(cv.tile_bytes - kStageOff - outlier_block_bytes(cv.n_out));
  for (int n = 0; n <= kMaxOutliers; ++n) {
    size_t sz = 0;
    attn_stages<BITS, NB>(plain + (uint32_t)outlier_block_bytes(n), n, &sz);
    cap = sz > cap ? sz : cap;
  }
  const cudaError_t e =
      cudaFuncSetAttribute(attn_kernel<BITS, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cap);
  if (e != cudaSuccess) return e;
  if (!a.pdl) {
    attn_kernel<BITS, NB><<<grid, 128, smem, st>>>(cv, a, lens);
    return cudaGetLastError();
  }
  // a programmatic dependent of the kernel before it on the stream
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(128);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, attn_kernel<BITS, NB>, cv, a, lens);
}

template <int NB>
cudaError_t launch_nb(const dim3& grid, const CacheView& cv, const AttnArgs& a, const SeqLens& lens,
                      cudaStream_t st) {
  switch (cv.bits) {
    case 2: return launch_bits<2, NB>(grid, cv, a, lens, st);
    case 3: return launch_bits<3, NB>(grid, cv, a, lens, st);
    case 4: return launch_bits<4, NB>(grid, cv, a, lens, st);
    default: return launch_bits<8, NB>(grid, cv, a, lens, st);
  }
}

}  // namespace

cudaError_t launch_wait_probe(int* status, cudaStream_t st) {
  wait_probe_kernel<<<1, 32, 0, st>>>(status);
  return cudaGetLastError();
}

cudaError_t launch_attention(const CacheView& cv, const AttnArgs& a, const SeqLens& lens, cudaStream_t st) {
  const int grp = a.Hq / cv.H;
  const int nhc = (grp + kNH - 1) / kNH;
  const dim3 grid(a.splits, cv.H * nhc, cv.B);
  return attn_key_blocks(grp) == 2 ? launch_nb<2>(grid, cv, a, lens, st) : launch_nb<1>(grid, cv, a, lens, st);
}

}  // namespace kivi
