// block_attention.cuh -- decode attention over listed packed blocks and the
// window (kAttnList, attention_blocks.cu), and over the whole cache with every
// block's softmax sum recorded (kAttnMass, attention_mass.cu).
//
// The packed tiles are those of attention.cuh, with the weights of the value
// product as fp16 pairs (bf16 lists: as there).  The window's tokens [t_tail, l) run on the tensor
// cores too: the rings' fp16 rows, and the rows that are already packed as
// fp16 pairs.
#pragma once

#include "attention.cuh"

namespace kivi {
namespace {

// ---------------------------------------------------------------------------
// The window, 32 tokens (one tile's) at a time:
//   S^T = q K^T   A: rows g = hi, g + 8 = lo of head g; B: warp w's tokens 8 w .. + 7
//   O   = P V     A: rows g = hi, g + 8 = lo of head g's weights; B: warp w's channels 32 w .. + 31
// Ring rows and packed blocks are staged by asynchronous copies; packed rows are
// dequantized (c * s + z) to fp16 pairs, a plane each, and ldmatrix takes the
// operands.  The scores pass through shared memory, and every warp takes the
// softmax of all 32 tokens.  The code runs once or twice a CTA, so it is bound
// by instruction fetch: loops stay rolled and nothing is specialized (a
// straight-line form of 2600 instructions a warp stalled 11 cycles an
// instruction for fetch, and took 19 us where this takes 6).

constexpr int kWinRow = kHeadDim + 8;    // halves of a row (rows 16 bytes apart in the banks)
constexpr int kWinX = kGroup + 4;        // floats of a head's scores
constexpr float kHalfMax = 65504.0f;

template <int BITS>
struct WinSmem {
  __half q[2][kNH][kWinRow];       // hi, lo of q * 2^-E
  __half k[2][kGroup][kWinRow];    // hi, lo of the keys
  __half v[2][kGroup][kWinRow];    // ... and values
  float x[kNH][kWinX];             // scores
  uint4 kc[kGroup * kRowBytes<BITS> / 16], vc[kGroup * kRowBytes<BITS> / 16];  // the tile's code rows
  uint32_t kg[2][64], vg[2][64];   // its scales and zeros
  uint32_t ko[outlier_block_bytes(kMaxOutliers) / 4];
  float ks[kNH];                   // 2^E * scale * log2(e)
  unsigned long long bar;          // completion of a round's copies
};

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}

// Eight floats as halves to hi, and what the halves leave of them to lo.  A
// dequantized value may exceed the fp16 range by its last rounding.
__device__ __forceinline__ void store_pair(const float (&v)[8], __half* hi, __half* lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = v[2 * i], b = v[2 * i + 1];
    h[i] = f2_to_h2(fminf(fmaxf(a, -kHalfMax), kHalfMax), fminf(fmaxf(b, -kHalfMax), kHalfMax));
    l[i] = f2_to_h2(a - h_lo(h[i]), b - h_hi(h[i]));
  }
  *reinterpret_cast<uint4*>(hi) = make_uint4(h[0], h[1], h[2], h[3]);
  *reinterpret_cast<uint4*>(lo) = make_uint4(l[0], l[1], l[2], l[3]);
}

// The codes of channels 8 x .. 8 x + 7 of a tile's key row r, as they lie
// there (3 bits: the low bits, then the high unit in the upper half).
template <int BITS>
__device__ __forceinline__ uint2 key_chunk(const uint8_t* rows, int r, int x) {
  const uint8_t* row = rows + r * kRowBytes<BITS>;
  if constexpr (BITS == 2) return make_uint2(*reinterpret_cast<const uint16_t*>(row + 2 * x), 0u);
  if constexpr (BITS == 3)
    return make_uint2(*reinterpret_cast<const uint16_t*>(row + 2 * x) |
                          (uint32_t)*reinterpret_cast<const uint16_t*>(row + kHiPlane3 + 4 * ((x >> 1) & 3) + 2 * (x & 1)) << 16,
                      0u);
  if constexpr (BITS == 4) return make_uint2(*reinterpret_cast<const uint32_t*>(row + 4 * x), 0u);
  return *reinterpret_cast<const uint2*>(row + krow_byte<8>(r, 8 * x));
}
// ... of value row r (two units of four channels; 3 bits: with their high units).
template <int BITS>
__device__ __forceinline__ uint2 value_chunk(const uint8_t* rows, int r, int x) {
  const uint8_t* row = rows + r * kRowBytes<BITS>;
  const int pos = 8 * (x & 3) + (x >> 2);  // of unit 2 x; the next at + 4
  if constexpr (BITS == 2) return make_uint2((uint32_t)row[pos] | (uint32_t)row[pos + 4] << 8, 0u);
  if constexpr (BITS == 3)
    return make_uint2((uint32_t)row[pos] | (uint32_t)row[pos + 4] << 8,
                      *reinterpret_cast<const uint32_t*>(row + kHiPlane3 + 4 * (x & 3)));
  if constexpr (BITS == 4)
    return make_uint2((uint32_t)*reinterpret_cast<const uint16_t*>(row + 2 * pos) |
                          (uint32_t)*reinterpret_cast<const uint16_t*>(row + 2 * pos + 8) << 16,
                      0u);
  return make_uint2(*reinterpret_cast<const uint32_t*>(row + vrow_byte<8>(r, 4 * pos)),
                    *reinterpret_cast<const uint32_t*>(row + vrow_byte<8>(r, 4 * pos + 16)));
}
// Code e of either chunk (value: the eight bits of a unit's high plane differ).
template <int BITS, bool VALUE>
__device__ __forceinline__ float chunk_code(uint2 w, int e, int x) {
  if constexpr (BITS == 8) return (float)(((e < 4 ? w.x : w.y) >> (8 * (e & 3))) & 255u);
  if constexpr (BITS == 4) return (float)((w.x >> (4 * e)) & 15u);
  uint32_t c = (w.x >> (2 * e)) & 3u;
  if constexpr (BITS == 3) {
    if constexpr (VALUE) {
      const int gp = x >> 2;
      c |= ((w.y >> (16 * (e >> 2) + hi_bit3(gp >> 1, 4 * (gp & 1) + (e & 3)))) & 1u) << 2;
    } else {
      c |= ((w.x >> (16 + hi_bit3(x >> 3, e))) & 1u) << 2;
    }
  }
  return (float)c;
}

// Scales or zeros of channels 8 x .. 8 x + 7 of a tile's key group, from the
// vector in its stored order (see kscale_pos), as four words of two channels
// in order.
template <int BITS>
__device__ __forceinline__ void key_params(const uint32_t* vec, int x, uint32_t (&w)[4]) {
  const uint4* v = reinterpret_cast<const uint4*>(vec);
  if constexpr (BITS <= 3) {
    // pair block x >> 1: word i holds channels 16 (x >> 1) + i and + 8
    const uint4 a = v[2 * (x >> 1)], b = v[2 * (x >> 1) + 1];
    const uint32_t sel = (x & 1) ? 0x7632u : 0x5410u;
    w[0] = __byte_perm(a.x, a.y, sel), w[1] = __byte_perm(a.z, a.w, sel);
    w[2] = __byte_perm(b.x, b.y, sel), w[3] = __byte_perm(b.z, b.w, sel);
  } else {
    // 4 bits: block x, word i channels 8 x + i and + 4; 8 bits: blocks 2 x and
    // 2 x + 1, word i channels 4 m + i and + 2
    const uint4 a = v[x];
    if constexpr (BITS == 4) {
      w[0] = __byte_perm(a.x, a.y, 0x5410), w[1] = __byte_perm(a.z, a.w, 0x5410);
      w[2] = __byte_perm(a.x, a.y, 0x7632), w[3] = __byte_perm(a.z, a.w, 0x7632);
    } else {
      w[0] = __byte_perm(a.x, a.y, 0x5410), w[1] = __byte_perm(a.x, a.y, 0x7632);
      w[2] = __byte_perm(a.z, a.w, 0x5410), w[3] = __byte_perm(a.z, a.w, 0x7632);
    }
  }
}

// The weights of a unit's blocks from its records and its heads' totals, by
// the CTA that has just merged the unit (see mass_kernel): its blocks are few,
// and a launch of its own would cost more than it computes.
__device__ __forceinline__ void fold_mass(const AttnArgs& a, long unit, int nh, int blocks,
                                          const float2 (&total)[kNH]) {
  const float* old = a.mass_in ? a.mass_in + unit * a.mass_row : nullptr;
#pragma unroll 1
  for (int i = threadIdx.x; i < a.mass_row; i += blockDim.x) {
    const float before = old ? a.decay * old[i] : 0.0f;
    float w = 0.0f;
    if (i < blocks) {
      const float4* rec = reinterpret_cast<const float4*>(a.records + (unit * a.record_blocks + i) * kNH);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (4 * half >= nh) break;
        const float4 r[2] = {__ldcg(rec + 2 * half), __ldcg(rec + 2 * half + 1)};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int j = 4 * half + 2 * k;
          if (j < nh) w += r[k].y * fast_exp2(r[k].x - total[j].x) / total[j].y;
          if (j + 1 < nh) w += r[k].w * fast_exp2(r[k].z - total[j + 1].x) / total[j + 1].y;
        }
      }
    }
    a.mass_out[unit * a.mass_row + i] = before + w;
  }
}

// A head's running softmax over the window and this lane's part of its
// output: head g, channels 32 warp + 8 i + 2 tig, + 1 in O[i][0] + O[i][2] and
// O[i][1] + O[i][3].
struct WinState {
  float m, l;
  float O[4][4];
};

// Tokens [first, end) for the CTA's heads, on top of `st` (m, l alike in the
// lanes of a head).  kAttnMass: the records of their blocks.
template <int BITS, int MODE>
__device__ __forceinline__ void window_tokens(const CacheView& cv, const AttnArgs& a, const SeqPlan& p,
                                              WinSmem<BITS>& ws, long unit, long gid, int b, int j0, int nh, int first,
                                              int end, WinState& st) {
  constexpr uint32_t kRows = kGroup * kRowBytes<BITS>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, tig = lane & 3;
  const int x = tid & 15, r0 = tid >> 4;  // this thread's channels 8 x .. + 7 and rows r0 + 8 i
  uint32_t parity = 0;
#pragma unroll 1
  for (int t0 = first; t0 < end; t0 += kGroup, parity ^= 1u) {
    const int n = min(kGroup, end - t0);
    const int nk = max(0, min(n, p.nq_k - t0)), nv = max(0, min(n, p.nq_v - t0));  // packed rows, in front
    const uint8_t* tile = tile_at<BITS>(cv, unit, t0 / kGroup);
    // ---- stage the round (the buffers were last used by ordinary accesses
    //      before a barrier): packed blocks by bulk copies of one thread, ring
    //      rows sixteen bytes a thread ----
    if (tid == 0) {
      const uint32_t ob = (uint32_t)outlier_block_bytes(cv.n_out);
      if (t0 == first) {
        mbar_init(&ws.bar, 1);
        mbar_fence_init();
      }
      mbar_expect_tx(&ws.bar, (nk ? kRows + 4 * kHeadDim + ob : 0u) + (nv ? kRows + 4 * kHeadDim : 0u));
      fence_proxy_async();
      if (nk) {
        bulk_g2s(ws.kc, tile + kOffKc<BITS>, kRows, &ws.bar);
        bulk_g2s(ws.kg[0], tile + kOffSk<BITS>, 2 * kHeadDim, &ws.bar);
        bulk_g2s(ws.kg[1], tile + kOffZk, 2 * kHeadDim, &ws.bar);
        if (ob) bulk_g2s(ws.ko, tile + kTileBytes<BITS>, ob, &ws.bar);
      }
      if (nv) {
        bulk_g2s(ws.vc, tile + kOffVc<BITS>, kRows, &ws.bar);
        bulk_g2s(ws.vg, tile + kOffSv<BITS>, 4 * kHeadDim, &ws.bar);
      }
    }
    {
      const int s0 = t0 % cv.W;  // (a round is no longer than the ring)
      const __half* rk = cv.ring_k + unit * cv.W * kHeadDim + 8 * x;
      const __half* rv = cv.ring_v + unit * cv.W * kHeadDim + 8 * x;
#pragma unroll
      for (int i = 0; i < kGroup / 8; ++i) {
        const int r = r0 + 8 * i, slot = s0 + r < cv.W ? s0 + r : s0 + r - cv.W;
        if (r >= nk && r < n) copy16(&ws.k[0][r][8 * x], rk + slot * kHeadDim);
        if (r >= nv && r < n) copy16(&ws.v[0][r][8 * x], rv + slot * kHeadDim);
      }
    }
    // ---- q, once: thread (head r0, channels 8 x .. + 7) ----
    if (t0 == first) {
      float v[8], amax = 0.0f;
      const long q0 = ((long)b * a.Hq + j0 + r0) * kHeadDim + 8 * x;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = r0 < nh ? load_q(a.q, q0 + i, a.q_dtype) : 0.0f;
        amax = fmaxf(amax, fabsf(v[i]));
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
      const int be = (int)((__float_as_uint(amax) >> 23) & 0xffu);
      const int E = amax == 0.0f ? 0 : (be == 0 ? -126 : be - 126);
      const float inv = ldexpf(1.0f, -E);  // |q| 2^-E < 1, exact
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= inv;
      store_pair(v, &ws.q[0][r0][8 * x], &ws.q[1][r0][8 * x]);
      if (x == 0) ws.ks[r0] = ldexpf(a.scale_log2, E);
      __syncthreads();  // the barrier is initialized (and q staged)
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!mbar_wait(&ws.bar, parity) && tid == 0) atomicOr(a.status, 1);

    // ---- packed rows to fp16 pairs; zeros where a product reads no row ----
    if (nk) {
      uint32_t sk[4], zk[4];
      key_params<BITS>(ws.kg[0], x, sk);
      key_params<BITS>(ws.kg[1], x, zk);
#pragma unroll 1
      for (int r = r0; r < kGroup; r += 8) {
        if (r < nk) {
          const uint2 c = key_chunk<BITS>(reinterpret_cast<const uint8_t*>(ws.kc), r, x);
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[e] = fmaf(chunk_code<BITS, false>(c, e, x), (e & 1) ? h_hi(sk[e >> 1]) : h_lo(sk[e >> 1]),
                        (e & 1) ? h_hi(zk[e >> 1]) : h_lo(zk[e >> 1]));
          store_pair(v, &ws.k[0][r][8 * x], &ws.k[1][r][8 * x]);
        } else {
          *reinterpret_cast<uint4*>(&ws.k[1][r][8 * x]) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      if (cv.n_out > 0) {
        // the fp16 outlier channels of the group (0 above): thread r takes row r
        __syncthreads();
        if (tid < nk) {
          const __half* ov = reinterpret_cast<const __half*>(&ws.ko[4]) + tid * cv.n_out;
          for (int o = 0; o < cv.n_out; ++o) ws.k[0][tid][(ws.ko[0] >> (8 * o)) & 0xffu] = ov[o];
        }
      }
    }
#pragma unroll 1
    for (int r = r0; r < kGroup; r += 8) {
      if (r < nv) {
        const uint2 c = value_chunk<BITS>(reinterpret_cast<const uint8_t*>(ws.vc), r, x);
        const int vs = vscale_pos(r, x >> 2);
        const float s = __half2float(reinterpret_cast<const __half*>(ws.vg[0])[vs]);
        const float z = __half2float(reinterpret_cast<const __half*>(ws.vg[1])[vs]);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(chunk_code<BITS, true>(c, e, x), s, z);
        store_pair(v, &ws.v[0][r][8 * x], &ws.v[1][r][8 * x]);
      } else {
        if (nv) *reinterpret_cast<uint4*>(&ws.v[1][r][8 * x]) = make_uint4(0u, 0u, 0u, 0u);
        if (r >= n) *reinterpret_cast<uint4*>(&ws.v[0][r][8 * x]) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    __syncthreads();

    // ---- scores of the warp's eight tokens ----
    {
      float S[4] = {0.f, 0.f, 0.f, 0.f};
      // ldmatrix rows: q plane (lane >> 3) & 1, head lane & 7, k half lane >> 4;
      // keys: token lane & 7, k quarter lane >> 3
      const __half* qp = &ws.q[(lane >> 3) & 1][lane & 7][8 * (lane >> 4)];
      const int krow = 8 * warp + (lane & 7), kcol = 8 * (lane >> 3);
#pragma unroll 1
      for (int c = 0; c < kHeadDim; c += 32) {
        uint32_t A0[4], A1[4], B[4];
        ldsm4(A0, qp + c);
        ldsm4(A1, qp + c + 16);
        ldsm4(B, &ws.k[0][krow][c + kcol]);
        mma16816(S, A0[0], A0[1], A0[2], A0[3], B[0], B[1]);
        mma16816(S, A1[0], A1[1], A1[2], A1[3], B[2], B[3]);
        if (nk) {
          ldsm4(B, &ws.k[1][krow][c + kcol]);
          mma16816(S, A0[0], A0[1], A0[2], A0[3], B[0], B[1]);
          mma16816(S, A1[0], A1[1], A1[2], A1[3], B[2], B[3]);
        }
      }
      const float ks = ws.ks[g];
      *reinterpret_cast<float2*>(&ws.x[g][8 * warp + 2 * tig]) = make_float2((S[0] + S[2]) * ks, (S[1] + S[3]) * ks);
    }
    __syncthreads();

    // ---- softmax of head g over tokens 2 tig + 8 i, + 1 (i < 4) ----
    float e[8];
    float mx = st.m;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 8 * i + 2 * tig;
      const float2 y = *reinterpret_cast<const float2*>(&ws.x[g][t]);
      e[2 * i] = t < n ? y.x : -INFINITY;
      e[2 * i + 1] = t + 1 < n ? y.y : -INFINITY;
      mx = fmaxf(mx, fmaxf(e[2 * i], e[2 * i + 1]));
    }
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));  // finite: the round holds a token
    const float corr = st.m == -INFINITY ? 0.0f : fast_exp2(st.m - mx);
    st.m = mx;
    float sum = 0.0f;
    uint32_t P[2][4];  // A of sixteen tokens: hi, lo of tokens 2 tig, + 1; hi, lo of + 8, + 9
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[2 * i] = fast_exp2(e[2 * i] - mx);
      e[2 * i + 1] = fast_exp2(e[2 * i + 1] - mx);
      sum += e[2 * i] + e[2 * i + 1];
      const uint32_t hi = f2_to_h2(e[2 * i], e[2 * i + 1]);
      P[i >> 1][2 * (i & 1)] = hi;
      P[i >> 1][2 * (i & 1) + 1] = f2_to_h2(e[2 * i] - h_lo(hi), e[2 * i + 1] - h_hi(hi));
    }
    sum += __shfl_xor_sync(kFull, sum, 1);
    sum += __shfl_xor_sync(kFull, sum, 2);
    st.l = st.l * corr + sum;
    if (MODE == kAttnMass && warp == 0 && tig == 0) *block_record(a, gid, t0 / kGroup, g) = make_float2(mx, sum);

    // ---- values of the warp's 32 channels ----
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) st.O[i][k] *= corr;
    // ldmatrix rows: token lane & 15, channel half lane >> 4
    const __half* vp = &ws.v[0][lane & 15][32 * warp + 8 * (lane >> 4)];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t B[4];
        ldsm4t(B, vp + 16 * kk * kWinRow + 16 * c);
        mma16816(st.O[2 * c], P[kk][0], P[kk][1], P[kk][2], P[kk][3], B[0], B[1]);
        mma16816(st.O[2 * c + 1], P[kk][0], P[kk][1], P[kk][2], P[kk][3], B[2], B[3]);
        if (nv) {
          ldsm4t(B, vp + (kGroup + 16 * kk) * kWinRow + 16 * c);
          mma16816(st.O[2 * c], P[kk][0], P[kk][1], P[kk][2], P[kk][3], B[0], B[1]);
          mma16816(st.O[2 * c + 1], P[kk][0], P[kk][1], P[kk][2], P[kk][3], B[2], B[3]);
        }
      }
    if (t0 + kGroup < end) __syncthreads();  // the rows are read
  }
}

// ---------------------------------------------------------------------------
// The packed tiles' q tables (PackedState), straight from a lane's channels:
// warp w takes heads w and w + 4, lane m channels 4 m .. 4 m + 3, whose halves
// go to their words (the words of build_q_tables).

// Channels 4 lane .. + 3 of the chunk's head j, zeros past the last head.
__device__ __forceinline__ float4 load_q4(const AttnArgs& a, int b, int j0, int nh, int j) {
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (j >= nh) return v;
  const long at = ((long)b * a.Hq + j0 + j) * kHeadDim + 4 * (threadIdx.x & 31);
  if (a.q_wide) {  // rows on a 16-byte boundary
    if (a.q_dtype == kF32) return *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + at);
    if (a.q_dtype == kF16) return make_float4(h_lo(w.x), h_hi(w.x), h_lo(w.y), h_hi(w.y));
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
  }
  v.x = load_q(a.q, at, a.q_dtype);
  v.y = load_q(a.q, at + 1, a.q_dtype);
  v.z = load_q(a.q, at + 2, a.q_dtype);
  v.w = load_q(a.q, at + 3, a.q_dtype);
  return v;
}

// 2^-E and 2^E * f for the least E with amax * 2^-E < 1 (subnormal and zero
// rows, and E past 126, as build_q_tables).
__device__ __forceinline__ void q_exponent(float amax, float f, float& inv, float& scale) {
  const int be = (int)((__float_as_uint(amax) >> 23) & 0xffu);
  const int E = amax == 0.0f ? 0 : (be == 0 ? -126 : be - 126);
  if (E <= 126) {
    inv = __uint_as_float((uint32_t)(127 - E) << 23);
  } else {
    inv = ldexpf(1.0f, -E);
  }
  scale = ldexpf(f, E);
}

// The packed splits' shared memory: one ring of `S` staged tiles of `stride`
// bytes for the CTA's warps (tile p of the split is in stage p mod S, and warp
// p mod 4 takes it), then this block, then q of the chunk's heads when the
// cache keeps outlier channels.  A ring that the warps share holds what a ring
// each would round away: 10 stages at 4 bits for 8, 11 at 8 bits for 8 (131k
// tokens at 4 bits: 48 us for 52; 128 units of 128 8-bit tiles: 38.7 for 41.1).
constexpr int kBetaRows = 16;   // tiles of a warp whose beta is held at once
constexpr int kRingMax = 24;    // stages at most

template <int NB>
struct BlockState : QTables<NB> {
  float beta[kWarps][kBetaRows][4 * NB];  // of the warp's tile k at row k mod kBetaRows
  unsigned long long bar[kRingMax];
  int issued[kRingMax];                   // copies issued into the stage so far
};

template <int BITS, int NB>
struct BlockView {
  unsigned char* base;
  int S;
  uint32_t stride;

  __device__ __forceinline__ TileBuf<BITS>& stage(int i) const {
    return *reinterpret_cast<TileBuf<BITS>*>(base + (size_t)i * stride);
  }
  __device__ __forceinline__ BlockState<NB>& ps() const {
    return *reinterpret_cast<BlockState<NB>*>(base + ((uint32_t)S * stride + 15u) / 16u * 16u);
  }
  __device__ __forceinline__ float* qo() const { return reinterpret_cast<float*>(&ps() + 1); }
  // a warp's output [kNH][kHeadDim], over the ring once every warp is done with it
  __device__ __forceinline__ float* merge_area(int w) const {
    return reinterpret_cast<float*>(base) + w * kNH * kHeadDim;
  }
};

template <int BITS, int NB, int MODE>
__device__ __forceinline__ void make_q_tables(const BlockView<BITS, NB>& sv, const AttnArgs& a, const float4 (&q4)[NB],
                                              bool keep_q) {
  BlockState<NB>& s = sv.ps();
  const int warp = threadIdx.x >> 5, m = threadIdx.x & 31;
  // channel 4 m + i sits in word wq + i (8 bits: wq + (i & 1)) of a quarter, as
  // its low or high half
  int tig, quarter, wq, half;
  if constexpr (BITS <= 3) tig = (m >> 2) & 3, quarter = 2 * (m >> 4) + (m & 1), wq = 0, half = (m >> 1) & 1;
  else if constexpr (BITS == 4) tig = (m >> 1) & 3, quarter = m >> 3, wq = 0, half = m & 1;
  else tig = m >> 3, quarter = (m & 7) >> 1, wq = 2 * (m & 1), half = 0;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int j = warp + kWarps * nb;
    const float v[4] = {q4[nb].x, q4[nb].y, q4[nb].z, q4[nb].w};
    const float amax = warp_max(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))));
    float inv, scale;
    q_exponent(amax, a.scale_log2, inv, scale);
    if (m == 0) s.qscale[j] = scale;
    if (keep_q) {
      const float sl = a.scale_log2;
      *reinterpret_cast<float4*>(sv.qo() + j * kHeadDim + 4 * m) = make_float4(v[0] * sl, v[1] * sl, v[2] * sl, v[3] * sl);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int w = BITS == 8 ? wq + (i & 1) : i, hf = BITS == 8 ? i >> 1 : half;
      // the channel's code position decides the table's scale
      const float f = BITS <= 3 && (m & 1) ? key_table_scale<BITS, MODE>((i + 4) & 7)
                                           : key_table_scale<BITS, MODE>(BITS == 8 ? 0 : i);
      const float x = v[i] * inv, y = x * f;
      const __half xh = __float2half_rn(x), yh = __float2half_rn(y);
      const __half xl = __float2half_rn(x - __half2float(xh)), yl = __float2half_rn(y - __half2float(yh));
      // the beta MMAs take words (0, 2) and (1, 3) of a quarter as B pairs
      const int wb = w == 1 ? 2 : (w == 2 ? 1 : w);
      auto put = [&](uint4 (&t)[4][8][4], int col, int word, __half h) {
        reinterpret_cast<__half*>(&t[quarter][col][tig])[2 * word + hf] = h;
      };
      if constexpr (NB == 1) {
        put(s.qs[0], 2 * j, w, yh);
        put(s.qs[1], 2 * j, w, __ushort_as_half(0));
        put(s.qs[0], 2 * j + 1, w, yl);
        put(s.qs[1], 2 * j + 1, w, yh);
        put(s.qb[0], 2 * j, wb, xh);
        put(s.qb[0], 2 * j + 1, wb, xl);
      } else {
        put(s.qs[0], j, w, yh);
        put(s.qs[1], j, w, yl);
        put(s.qb[0], j, wb, xh);
        put(s.qb[NB - 1], j, wb, xl);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Waits, bounded, until turn `turn` of a stage has landed.  The warps share the
// ring, and the copy of a turn is issued by the warp that was done with the
// turn before: `issued` says that this has happened, which the barrier's parity
// alone cannot (two turns back looks the same).
__device__ __forceinline__ bool stage_wait(unsigned long long* bar, const int* issued, int turn) {
  const volatile int* count = issued;
  if (*count > turn && mbar_try_wait(bar, turn & 1)) return true;
  const unsigned long long t0 = global_ns();
  while (*count <= turn) {
    if (global_ns() - t0 > kWaitLimitNs) return false;
  }
  return mbar_wait(bar, turn & 1);
}

// Packed tiles: positions [tile0, tile1) of the unit's list (kAttnList) or of
// its tiles, as attention.cu's packed_split, in one loop whose body holds each
// part once (a list may give a warp two tiles: a part that is unrolled for the
// first or the last one costs its instruction fetch).
template <int BITS, int NB, int MODE>
__device__ __forceinline__ void packed_blocks_split(const CacheView& cv, const AttnArgs& a, const BlockView<BITS, NB>& sv,
                                                    long unit, long gid, int b, int j0, int nh, int tile0, int tile1,
                                                    int blocks, float (&s_m)[kWarps][kNH], float (&s_l)[kWarps][kNH]) {
  const int S = sv.S;
  BlockState<NB>& ws = sv.ps();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, tig = lane & 3;
  const int n = tile1 - tile0;                                    // the CTA's tiles
  const int n_mine = n > warp ? (n - warp + kWarps - 1) / kWarps : 0;  // this warp's: warp, warp + 4, ...
  const float* const qo = sv.qo();
  const UnitSrc us = unit_src<BITS>(cv, a, unit, blocks);
  // the tile at position p of the split (an entry that names no block: tile 0,
  // staged in its place and left out of the softmax)
  auto entry = [&](int p) { return attn_listed(MODE) ? us.list[tile0 + p] : tile0 + p; };
  // lane k: the entry of the warp's tile 32 block + k
  auto my_entry = [&](int block) {
    const int k = 32 * block + lane;
    return k < n_mine ? entry(warp + kWarps * k) : -1;
  };
  int id = 0;
  uint4 z[2][4];
  auto load_z = [&](int k0) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int k = k0 + g + 8 * r;
      const int e = __shfl_sync(kFull, id, k & 31);
      const uint4* v = reinterpret_cast<const uint4*>(us.tiles + (long)us.tile(e) * us.stride + kOffZk);
#pragma unroll
      for (int q = 0; q < 4; ++q) z[r][q] = k < n_mine ? __ldg(v + zk_chunk<BITS>(tig, q)) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  // the first copies and the key zeros go out before the q tables are built; a
  // launch whose list the launch before it writes waits for that first.
  // (Lane i of warp w owns stage w + 4 i: it initializes the stage's barrier
  // and issues its first tile, a quarter of the copies a warp, one at a time.)
  const int p0 = warp + kWarps * lane;
  auto begin = [&]() {
    if (p0 < min(n, S)) {
      ws.issued[p0] = 1;
      issue_tile<BITS>(sv.stage(p0), &ws.bar[p0], us, us.tile(id));
    }
    __syncwarp();
    load_z(0);
  };
  const bool wait_late = a.pdl == kPdlAll;
  if (!wait_late) id = my_entry(0);
  float4 q4[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) q4[nb] = load_q4(a, b, j0, nh, warp + kWarps * nb);
  if (p0 < S) {
    mbar_init(&ws.bar[p0], 1);
    mbar_fence_init();
  }
  if (!wait_late) begin();
  make_q_tables<BITS, NB, MODE>(sv, a, q4, cv.n_out > 0);
  if (wait_late) {
    grid_dependency_wait();
    id = my_entry(0);
    begin();
  }
  __syncthreads();
  float* const brows = &ws.beta[warp][0][0];
  beta_mma<NB>(ws, z, g, tig, brows);
  __syncwarp();
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
  uint32_t pb[2][2], pl[2][2];  // the weights of the tile before (see softmax_p)
  float ts[NB];
  int sk = warp, sp = 0;  // the stages of tiles k and k - 1 (S > kWarps)
  int turn = 0, tp = 0;   // ... and their turns there
  bool failed = false;
#pragma unroll 1
  for (int k = 0; n_mine > 0; ++k) {
    float sc[NB][4];
    bool live = k < n_mine;
    const int pn = warp + kWarps * (k - 1) + S;  // the tile that follows in the stage of tile k - 1
    const bool more = k > 0 && pn < n;
    const int next = more ? entry(pn) : 0;
    if (live) {
      // a position that names no block adds nothing
      if (attn_listed(MODE)) live = (unsigned)__shfl_sync(kFull, id, k & 31) < (unsigned)blocks;
      if (__any_sync(kFull, !stage_wait(&ws.bar[sk], &ws.issued[sk], turn))) {
        failed = true;
        break;
      }
      if (k % kBetaRows == 0 && k > 0) {
        // beta of the next sixteen tiles
        __syncwarp();
        load_z(k);
        beta_mma<NB>(ws, z, g, tig, brows);
        __syncwarp();
      }
      float mb[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mb[nb] = m_run[nb] == -INFINITY ? 0.0f : m_run[nb];
      key_scores<BITS, NB, MODE>(ws, sv.stage(sk), g, tig, ks, mb, cv.n_out, qo, brows + (k % kBetaRows) * 4 * NB, sc);
    }
    if (k > 0) {
      value_acc<BITS, NB, MODE>(sv.stage(sp), pb, pl, g, tig, O, Z);
      __syncwarp();  // every lane is done with the stage
      if (more && lane == 0) *const_cast<volatile int*>(&ws.issued[sp]) = tp + 2;
      issue_tile_if<BITS>(more && lane == 0, sv.stage(sp), &ws.bar[sp], us.tiles + (long)us.tile(next) * us.stride + kStageOff,
                          us.copy);
    }
    if (k >= n_mine) break;
    if (live) {
      softmax_p<BITS, NB, MODE>(sc, g, tig, m_run, O, Z, pb, pl, ts);
      if constexpr (MODE == kAttnMass) {
        // the record (running max, sum) of the tile, one lane per head
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float v = ts[nb];
          v += __shfl_xor_sync(kFull, v, 4);
          v += __shfl_xor_sync(kFull, v, 8);
          v += __shfl_xor_sync(kFull, v, 16);
          if (g == 0)
            *block_record(a, gid, tile0 + warp + kWarps * k, NB == 1 ? tig : 2 * tig + nb) = make_float2(m_run[nb], v);
        }
      }
    } else {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        pb[kk][0] = pb[kk][1] = 0u;
        if constexpr (attn_pairs(MODE)) pl[kk][0] = pl[kk][1] = 0u;
      }
      // tile 0 in its place may hold anything, and its weights are zeros: so are
      // the value scales and zeros (256 listed tiles of 8 units, no hole among
      // them: 10.1 us so, 10.3 where the value product is skipped)
      if constexpr (attn_listed(MODE)) {
        reinterpret_cast<uint4*>(sv.stage(sk).sv)[lane] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async();  // (a bulk copy follows in the stage)
        __syncwarp();
      }
    }
    sp = sk, tp = turn;
    sk += kWarps;
    if (sk >= S) sk -= S, ++turn;
    if ((k & 31) == 31) id = my_entry((k >> 5) + 1);
  }
  // the ring is free once every warp is done with it (the merge areas and the
  // window take its memory)
  if (__syncthreads_or(failed)) {
    // A wait timed out: record it, and let the copies still in flight land
    // (each wait bounded again).
    if (tid == 0) atomicOr(a.status, 1);
    if (tid < min(n, S)) mbar_wait(&ws.bar[tid], (uint32_t)(ws.issued[tid] - 1) & 1u);
    __syncthreads();
  }
  if (tid < S) mbar_inval(&ws.bar[tid]);

  // the lo parts' columns 4..7 join columns 0..3
  if constexpr (NB == 1 && attn_pairs(MODE)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Z[i] += __shfl_xor_sync(kFull, Z[i], 2);
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) O[mt][i] += __shfl_xor_sync(kFull, O[mt][i], 2);
    }
  }
  // ---- this warp's partial: max, sum and output per head (as packed_split) ----
  if (g == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (NB == 2) s_m[warp][2 * tig + i] = m_run[i];
      else s_m[warp][4 * i + tig] = i == 0 ? m_run[0] : -INFINITY;
    }
    s_l[warp][2 * tig] = Z[2];
    s_l[warp][2 * tig + 1] = Z[3];
  }
  float zt[4][2];
#pragma unroll
  for (int gp = 0; gp < 4; ++gp) {
    zt[gp][0] = __shfl_sync(kFull, Z[0], 4 * gp + tig);
    zt[gp][1] = __shfl_sync(kFull, Z[1], 4 * gp + tig);
  }
  if (n_mine == 0 || (NB == 1 && tig >= 2)) return;  // (columns 4..7: joined above, or heads 0..3 again)
  float* oa = sv.merge_area(warp) + (2 * tig) * kHeadDim;
  float* ob = oa + kHeadDim;
#pragma unroll
  for (int mt = 0; mt < 8; ++mt) {
    const int gp = mt >> 1, hm = mt & 1;
    const int i_lo = BITS <= 3 ? 4 * (gp & 1) + 2 * hm : 2 * hm;
    const int ch = 32 * gp + 4 * g + 2 * hm;
    const float f_lo = value_unit<BITS, MODE>(i_lo), f_hi = value_unit<BITS, MODE>(i_lo + 1);
    oa[ch] = O[mt][0] * f_lo + zt[gp][0];
    ob[ch] = O[mt][1] * f_lo + zt[gp][1];
    oa[ch + 1] = O[mt][2] * f_hi + zt[gp][0];
    ob[ch + 1] = O[mt][3] * f_hi + zt[gp][1];
  }
}

__device__ __forceinline__ void store_out(const AttnArgs& a, long i, float x) {
  if (a.q_dtype == kF32) static_cast<float*>(a.out)[i] = x;
  else if (a.q_dtype == kF16) static_cast<__half*>(a.out)[i] = __float2half_rn(x);
  else static_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16_rn(x);
}

// Merges n <= 64 partials of the warp's heads (warp, and with two key blocks
// warp + 4), lane l channels 4 l .. 4 l + 3, sixteen loads at once.
static_assert(kFlatMerge == 64 && kMergeGroup <= 32, "two partials a lane");

template <int NB>
__device__ __forceinline__ void merge_splits(const float* po, const float* pml, int n, float4 (&o4)[NB], float (&m)[NB],
                                             float (&l)[NB]) {
  constexpr int kAtOnce = 16 / NB;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float2 ml[NB][2];  // of partials lane, lane + 32
  float e[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      ml[nb][i] = lane + 32 * i < n
                      ? __ldcg(reinterpret_cast<const float2*>(pml + ((long)(lane + 32 * i) * kNH + warp + kWarps * nb) * 2))
                      : make_float2(-INFINITY, 0.0f);
    o4[nb] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float4* src = reinterpret_cast<const float4*>(po + (long)warp * kHeadDim) + lane;
#pragma unroll 1
  for (int k0 = 0; k0 < n; k0 += kAtOnce) {
    float4 v[NB][kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        v[nb][k] = k0 + k < n ? __ldcg(src + ((long)(k0 + k) * kNH + kWarps * nb) * (kHeadDim / 4))
                              : make_float4(0.f, 0.f, 0.f, 0.f);
    if (k0 == 0) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        m[nb] = warp_max(fmaxf(ml[nb][0].x, ml[nb][1].x));
#pragma unroll
        for (int i = 0; i < 2; ++i) e[nb][i] = ml[nb][i].x == -INFINITY ? 0.0f : fast_exp2(ml[nb][i].x - m[nb]);
        l[nb] = warp_sum(e[nb][0] * ml[nb][0].y + e[nb][1] * ml[nb][1].y);
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        // (0 past the last: ml is -inf there)
        const float ek = __shfl_sync(kFull, k0 < 32 ? e[nb][0] : e[nb][1], (k0 + k) & 31);
        o4[nb].x = fmaf(ek, v[nb][k].x, o4[nb].x);
        o4[nb].y = fmaf(ek, v[nb][k].y, o4[nb].y);
        o4[nb].z = fmaf(ek, v[nb][k].z, o4[nb].z);
        o4[nb].w = fmaf(ek, v[nb][k].w, o4[nb].w);
      }
  }
}

// 128 threads a CTA; the window's splits and the packed ones (SeqPlan) of every
// (batch, kv-head, head chunk), merged as attn_kernel's.  CTAs that all run at
// once come unit by unit, the window's first: grid (splits, H * head_chunks, B).
// Of more, every unit's packed splits start before the windows, as the longer
// ones (window_last): grid (H * head_chunks, B, splits).  128 units of 128 8-bit
// tiles (384 CTAs for 304 places) take 33.2 us so, 37.1 unit by unit; 8 units of
// 256 tiles 10.5 us so, 10.3 unit by unit.
// The next launch starts when this one has completed (attention calls with the
// overlap on read its output without waiting), the weights' launch of the same
// call (mass_kernel) too: 49.0 us for 131k tokens, as if it were let in earlier.
template <int BITS, int NB, int MODE>
__global__ void __launch_bounds__(128, attn_ctas_per_sm(BITS, NB))
    block_attn_kernel(CacheView cv, AttnArgs a, const SeqLens lens) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const BlockView<BITS, NB> sv{smem_raw, a.stages, (uint32_t)(cv.tile_bytes - kStageOff)};
  __shared__ float s_m[kWarps][kNH], s_l[kWarps][kNH];  // the packed tiles' partials
  __shared__ bool s_last;
  __shared__ float2 s_total[kNH];  // kAttnMass: the merged (max, sum) of every head

  const int z = a.window_last ? blockIdx.z : blockIdx.x;
  const int y = a.window_last ? blockIdx.x : blockIdx.y;
  const int b = a.window_last ? blockIdx.y : blockIdx.z;
  const int h = a.nhc == 1 ? y : y / a.nhc;
  const int hc = a.nhc == 1 ? 0 : y % a.nhc;
  const long gid = (long)b * (cv.H * a.nhc) + y;  // (batch, kv-head, head chunk)
  const int j0 = h * a.grp + hc * kNH;
  const int nh = min(kNH, a.grp - hc * kNH);
  const long unit = (long)b * cv.H + h;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SeqPlan p = lens.uniform >= 0
                        ? a.plan
                        : make_plan(lens.l[b], cv.R, cv.policy, a.scfg, attn_listed(MODE) ? a.list_len : -1);
  const int zt = a.window_last ? z + p.tail_splits : z;
  const int s = zt < p.splits ? zt : zt - p.splits;
  // Every launch starts as the one before it ends, and waits for it before it
  // touches memory.  kPdlAll (its list comes from the launch before it, its q and
  // cache from earlier ones): the packed splits wait after their q tables, the
  // window's at their end.
  const bool wait_late = a.pdl == kPdlAll && z < p.splits;
  if (!wait_late) {
    grid_dependency_wait();
  }
  if (z >= p.splits) return;
  const bool packed = s >= p.tail_splits;
  const bool window = !packed || (p.tail_fused && s == p.splits - 1);
  const bool only = p.splits == 1;
  if (packed) {
    const int sp = s - p.tail_splits;
    const int tile0 = sp * p.chunk / 32;
    const int tile1 = min(p.tiles, (sp + 1) * p.chunk / 32);
    packed_blocks_split<BITS, NB, MODE>(cv, a, sv, unit, gid, b, j0, nh, tile0, tile1, p.t_tail / kGroup, s_m, s_l);
    __syncthreads();
    // merge the warps' partials: warp w heads w and w + 4, lane l channels 4 l .. 4 l + 3
    float* fuse = reinterpret_cast<float*>(&sv.ps());  // the merged partial that the window goes on from
#pragma unroll 1
    for (int j = warp; j < nh; j += kWarps) {
      float mw[kWarps], M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        mw[w] = s_m[w][j];
        M = fmaxf(M, mw[w]);
      }
      float lt = 0.0f;
      float4 ot = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (mw[w] == -INFINITY) continue;  // no tile (its area is not written)
        const float e = fast_exp2(mw[w] - M);
        const float4 o = reinterpret_cast<const float4*>(sv.merge_area(w) + j * kHeadDim)[lane];
        lt += e * s_l[w][j];
        ot.x += e * o.x;
        ot.y += e * o.y;
        ot.z += e * o.z;
        ot.w += e * o.w;
      }
      if (window) {
        reinterpret_cast<float4*>(fuse + j * kHeadDim)[lane] = ot;
        if (lane < 2) fuse[(kNH + lane) * kHeadDim + j] = lane ? lt : M;
      } else {
        const long pidx = (gid * a.scfg.max_splits + s) * kNH + j;
        reinterpret_cast<float4*>(a.ws_o + pidx * kHeadDim)[lane] = ot;
        if (lane == 0) *reinterpret_cast<float2*>(a.ws_ml + pidx * 2) = make_float2(M, lt);
      }
    }
  }
  if (window) {
    const int g = lane >> 2, tig = lane & 3;
    WinState st;
    st.m = -INFINITY, st.l = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) st.O[i][k] = 0.0f;
    if (packed) {
      __syncthreads();
      const float* fuse = reinterpret_cast<const float*>(&sv.ps());
      if (g < nh) {
        st.m = fuse[kNH * kHeadDim + g];
        st.l = fuse[(kNH + 1) * kHeadDim + g];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 o = *reinterpret_cast<const float2*>(fuse + g * kHeadDim + 32 * warp + 8 * i + 2 * tig);
          st.O[i][0] = o.x, st.O[i][1] = o.y;
        }
      }
      __syncthreads();  // the partial is read; the window takes its memory
    }
    const int c0 = packed ? p.t_tail : p.t_tail + s * kTailTok;
    window_tokens<BITS, MODE>(cv, a, p, *reinterpret_cast<WinSmem<BITS>*>(smem_raw), unit, gid, b, j0, nh, c0,
                              packed ? p.l : min(p.l, c0 + kTailTok), st);
    if (wait_late && !packed) grid_dependency_wait();
    if (g < nh) {
      const float inv = only ? 1.0f / st.l : 1.0f;
      const long pidx = (gid * a.scfg.max_splits + s) * kNH + g;
      const long oi = ((long)b * a.Hq + j0 + g) * kHeadDim + 32 * warp + 2 * tig;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float o0 = (st.O[i][0] + st.O[i][2]) * inv, o1 = (st.O[i][1] + st.O[i][3]) * inv;
        if (only) {
          store_out(a, oi + 8 * i, o0);
          store_out(a, oi + 8 * i + 1, o1);
        } else {
          *reinterpret_cast<float2*>(a.ws_o + pidx * kHeadDim + 32 * warp + 8 * i + 2 * tig) = make_float2(o0, o1);
        }
      }
      if (warp == 0 && tig == 0) {
        if (only) {
          if (MODE == kAttnMass) {
            s_total[g] = make_float2(st.m, st.l);
            a.totals[gid * kNH + g] = make_float2(st.m, st.l);
          }
        } else {
          *reinterpret_cast<float2*>(a.ws_ml + pidx * 2) = make_float2(st.m, st.l);
        }
      }
    }
  }
  const int blocks = (p.l + kGroup - 1) / kGroup;
  if (only) {
    if (MODE == kAttnMass && a.fold) {
      __syncthreads();  // the records and totals are written
      fold_mass(a, unit, nh, blocks, s_total);
    }
    return;
  }

  // ---- the last CTA of a group of splits merges the group (up to 64 splits:
  //      one group; more: groups of kMergeGroup, whose results the last group
  //      merges) ----
  const int gs = p.splits <= kFlatMerge ? kFlatMerge : kMergeGroup;
  const int n_grp = (p.splits + gs - 1) / gs;
  const int grp_i = s / gs;
  const int g_lo = grp_i * gs, g_n = min(gs, p.splits - g_lo);
  __syncthreads();
  if (threadIdx.x == 0) {
    int* counter = a.counters + gid * a.merge_groups + grp_i;
    s_last = count_in(counter) == g_n - 1;
    if (s_last) *counter = 0;  // every other CTA of the group has counted in
  }
  __syncthreads();
  if (!s_last) return;
  // warp w merges heads w and, with two key blocks, w + kWarps (heads past the
  // chunk's last: their slots hold nothing that is used)
  float4 o4[NB];
  float lsum_h[NB], m_h[NB];
  merge_splits<NB>(a.ws_o + (gid * a.scfg.max_splits + g_lo) * kNH * kHeadDim,
                   a.ws_ml + (gid * a.scfg.max_splits + g_lo) * kNH * 2, g_n, o4, m_h, lsum_h);
  if (n_grp > 1) {
#pragma unroll
    for (int hh = 0; hh < NB; ++hh) {
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
    merge_splits<NB>(a.ws_o1 + gid * a.merge_groups * kNH * kHeadDim, a.ws_ml1 + gid * a.merge_groups * kNH * 2, n_grp, o4,
                     m_h, lsum_h);
  }
#pragma unroll
  for (int hh = 0; hh < NB; ++hh) {
    const int j = warp + kWarps * hh;
    if (j >= nh) continue;
    if (MODE == kAttnMass && lane == 0) {
      s_total[j] = make_float2(m_h[hh], lsum_h[hh]);
      a.totals[gid * kNH + j] = make_float2(m_h[hh], lsum_h[hh]);
    }
    const float inv = 1.0f / lsum_h[hh];
    const float r[4] = {o4[hh].x * inv, o4[hh].y * inv, o4[hh].z * inv, o4[hh].w * inv};
    const long oi = ((long)b * a.Hq + j0 + j) * kHeadDim + 4 * lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) store_out(a, oi + i, r[i]);
  }
  if (MODE == kAttnMass && a.fold) {
    __syncthreads();
    fold_mass(a, unit, nh, blocks, s_total);
  }
}

// Stages of a CTA's ring: as many as attn_ctas_per_sm CTAs per SM leave room
// for, and its dynamic shared memory.
constexpr size_t ring_stride(int bits, int n_out) {
  return (size_t)(2 * kGroup * (kHeadDim * bits / 8) + 8 * kHeadDim - kStageOff + outlier_block_bytes(n_out));
}
template <int NB>
constexpr size_t ring_fixed(int n_out) {
  return sizeof(BlockState<NB>) + (n_out > 0 ? (size_t)kNH * kHeadDim * 4 : 0) + 16;
}
template <int BITS, int NB>
constexpr int ring_room(int n_out) {
  const size_t per_cta = (size_t)228 * 1024 / attn_ctas_per_sm(BITS, NB) - 1024 - 512;
  return (int)((per_cta - ring_fixed<NB>(n_out)) / ring_stride(BITS, n_out));
}
template <int BITS, int NB>
int ring_stages(int n_out, size_t* smem) {
  static_assert(ring_stride(BITS, 0) == kTileBytes<BITS> - kStageOff, "a stage is a tile but for its key zeros");
  // (with kWarps stages a warp's tile would wait for the copy that only the end
  // of its tile before, in the same stage, lets go out)
  static_assert(ring_room<BITS, NB>(0) > kWarps && ring_room<BITS, NB>(1) > kWarps && ring_room<BITS, NB>(2) > kWarps &&
                    ring_room<BITS, NB>(3) > kWarps && ring_room<BITS, NB>(kMaxOutliers) > kWarps,
                "a stage more than warps");
  const size_t stride = ring_stride(BITS, n_out), fixed = ring_fixed<NB>(n_out);
  const int S = ring_room<BITS, NB>(n_out) < kRingMax ? ring_room<BITS, NB>(n_out) : kRingMax;
  const size_t packed = (S * stride + 15) / 16 * 16 + fixed;
  *smem = packed > sizeof(WinSmem<BITS>) ? packed : sizeof(WinSmem<BITS>);
  return S;
}

template <int BITS, int NB, int MODE>
cudaError_t launch_block_bits(const CacheView& cv, AttnArgs a, const SeqLens& lens, cudaStream_t st) {
  static_assert(attn_ctas_per_sm(BITS, NB) * (sizeof(WinSmem<BITS>) + 1024 + 512) <= 228 * 1024,
                "the window's layout fits the CTAs of an SM");
  static_assert(sizeof(QTables<NB>) >= (kNH + 2) * kHeadDim * 4, "the merged partial fits the q tables");
  size_t smem = 0, cap = 0;
  a.stages = ring_stages<BITS, NB>(cv.n_out, &smem);
  const int units = cv.H * a.nhc;
  const long ctas = (long)units * cv.B * a.splits, places = (long)attn_ctas_per_sm(BITS, NB) * kTargetSMs;
  a.window_last = ctas > places;
  // (the opt-in as in launch_bits: the same on every call)
  for (int n = 0; n <= kMaxOutliers; ++n) {
    size_t sz = 0;
    ring_stages<BITS, NB>(n, &sz);
    cap = sz > cap ? sz : cap;
  }
  const cudaError_t e = cudaFuncSetAttribute(block_attn_kernel<BITS, NB, MODE>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cap);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = a.window_last ? dim3(units, cv.B, a.splits) : dim3(a.splits, units, cv.B);
  lc.blockDim = dim3(128);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, block_attn_kernel<BITS, NB, MODE>, cv, a, lens);
}

template <int NB, int MODE>
cudaError_t launch_block_nb(const CacheView& cv, const AttnArgs& a, const SeqLens& lens,
                            cudaStream_t st) {
  switch (cv.bits) {
    case 2: return launch_block_bits<2, NB, MODE>(cv, a, lens, st);
    case 3: return launch_block_bits<3, NB, MODE>(cv, a, lens, st);
    case 4: return launch_block_bits<4, NB, MODE>(cv, a, lens, st);
    default: return launch_block_bits<8, NB, MODE>(cv, a, lens, st);
  }
}

template <int MODE>
cudaError_t launch_block_attention(const CacheView& cv, const AttnArgs& a, const SeqLens& lens, cudaStream_t st) {
  return attn_key_blocks(a.grp) == 2 ? launch_block_nb<2, MODE>(cv, a, lens, st)
                                     : launch_block_nb<1, MODE>(cv, a, lens, st);
}

}  // namespace
}  // namespace kivi
