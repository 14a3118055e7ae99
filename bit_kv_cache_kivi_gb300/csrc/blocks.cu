// blocks.cu -- operators on the packed blocks (32-token tiles) of a cache:
// an upper bound of q.k per block, the choice of the best blocks, the blocks'
// attention weights, and the eviction of blocks.
#include "kivi_internal.cuh"

namespace kivi {
namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float load_q(const void* q, long idx, int dt) {
  if (dt == kF32) return static_cast<const float*>(q)[idx];
  if (dt == kF16) return __half2float(static_cast<const __half*>(q)[idx]);
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(q)[idx] << 16);
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
  return v;
}

// ---------------------------------------------------------------------------
// Block scores.
//
// The keys of channel c of a block lie in [z_c, z_c + L s_c], L = 2^bits - 1,
// so no token of the block has a larger q.k than
//   sum_c max(q_c z_c, q_c (z_c + L s_c)) = sum_c q_c z_c + sum_c (L max(q_c, 0)) s_c,
// a product of the tile's 256 stored halves (zeros, scales) with a vector made
// of q: two 256-byte reads of a tile and no code.  Sixteen tiles are the rows
// of an m16n8k16 product as they are stored (the k order is the stored channel
// order, the table of q follows it), four query heads its columns as fp16 hi /
// lo pairs (q to about 2^-22, as the attention's tables).  fp16 outlier
// channels (their zeros and scales are 0) add the largest of their exact
// products over the block's tokens.
//
// Bound by latency, then by the loads: every load of a warp's sixteen tiles (8
// KB) is in flight at once, four CTAs an SM.  131k tokens of 8 units at 2 bits
// take 3.9 us (16.8 MB, 4.3 TB/s; one block row of 4097 tokens 2.3 us), 16
// sequences of up to 32k tokens, 4 KV heads of seven query heads, at 4 bits
// 7.3 us (24 MB).

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kScoreWarps = 4;
constexpr int kScoreTiles = 16 * kScoreWarps;  // tiles of a CTA
constexpr int kScoreHeads = 2 * kScoreWarps;   // query heads of a round: warp w makes the tables of w and w + 4

// Channels 4 lane .. + 3 of query head `head`.
__device__ __forceinline__ float4 load_q4(const void* q, long head, int dt, bool wide) {
  const long at = head * kHeadDim + 4 * (threadIdx.x & 31);
  if (wide && dt != kF32) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(q) + at);
    if (dt == kBF16)
      return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                         __uint_as_float(w.y & 0xffff0000u));
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
    const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
    return make_float4(lo.x, lo.y, hi.x, hi.y);
  }
  return make_float4(load_q(q, at, dt), load_q(q, at + 1, dt), load_q(q, at + 2, dt), load_q(q, at + 3, dt));
}

template <int BITS>
__global__ void __launch_bounds__(32 * kScoreWarps)
    score_kernel(CacheView cv, const void* q, int q_dtype, int q_wide, int grp, float* scores, int row, int release,
                 const SeqLens lens) {
  constexpr float L = (float)((1 << BITS) - 1);
  // the B fragments of a round's heads, four a block: [block][zeros, scales][16-byte chunk group][lane]
  __shared__ uint4 table[2][2][4][32];
  __shared__ float qs[kScoreHeads][kHeadDim];  // q * 2^-E of the heads (outlier channels only)
  __shared__ float2 qpow[kScoreHeads];         // 2^E, |q| 2^-E < 1, as two factors (E up to 128)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tig = lane & 3;
  const int h = blockIdx.y, b = blockIdx.z;
  const int nb = packed_blocks(seq_len(lens, b), cv.R, cv.policy);
  const long unit = (long)b * cv.H + h;
  const uint8_t* tiles = tile_at<BITS>(cv, unit, 0);
  float* out = scores + unit * row;
  grid_dependency_wait();
  if (release) grid_launch_dependents();
  // q of the first round before the tiles (the tables are made while those load)
  float4 q4[2];
  auto load_heads = [&](int j0) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int j = j0 + warp + 4 * k;
      q4[k] = j < grp ? load_q4(q, ((long)b * cv.H + h) * grp + j, q_dtype, q_wide) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  load_heads(0);
  // a grid of one wave: a CTA takes every gridDim.x-th group of 64 tiles, and
  // makes the tables once when one round holds the heads
  bool made = false;
#pragma unroll 1
  for (int at = blockIdx.x * kScoreTiles; at < row; at += gridDim.x * kScoreTiles) {
    if (at >= nb) {  // the row behind the last block
      const int j = at + threadIdx.x;
      if (threadIdx.x < kScoreTiles && j < row) out[j] = -INFINITY;
      continue;
    }
    const int t0 = at + 16 * warp;  // this warp's tiles
    // A: rows g and g + 8; chunk group c of lane tig is the 16-byte chunk 4 c + tig
    uint4 a[2][2][4];  // [row half][zeros, scales][chunk group]
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int t = t0 + g + 8 * r;
      const uint4* z = reinterpret_cast<const uint4*>(tiles + (long)t * cv.tile_bytes + kOffZk);
      const uint4* s = reinterpret_cast<const uint4*>(tiles + (long)t * cv.tile_bytes + kOffSk<BITS>);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        a[r][0][c] = t < nb ? __ldg(z + 4 * c + tig) : make_uint4(0u, 0u, 0u, 0u);
        a[r][1][c] = t < nb ? __ldg(s + 4 * c + tig) : make_uint4(0u, 0u, 0u, 0u);
      }
    }

    float best0 = -INFINITY, best1 = -INFINITY;  // of tiles t0 + g, t0 + g + 8
#pragma unroll 1
    for (int j0 = 0; j0 < grp; j0 += kScoreHeads) {
      const int blocks = grp - j0 > 4 ? 2 : 1;
      if (!made || grp > kScoreHeads) {
        if (made) {
          load_heads(j0);
          __syncthreads();  // the tables of the heads before are read
        }
        made = true;
        // ---- tables: warp w heads j0 + w and j0 + w + 4, lane channels 4 lane .. + 3,
        //      scaled by a power of two; a channel's halves go to its stored slot ----
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (k >= blocks) break;
          float v[4] = {q4[k].x, q4[k].y, q4[k].z, q4[k].w};
          const float amax = warp_max(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))));
          const int be = (int)((__float_as_uint(amax) >> 23) & 0xffu);
          const int E = amax == 0.0f ? 0 : (be == 0 ? -126 : be - 126);
          // exact: powers of two (2^-E subnormal for E > 126)
          const float inv = E <= 126 ? __uint_as_float((uint32_t)(127 - E) << 23) : ldexpf(1.0f, -E);
          if (lane == 0) qpow[warp + 4 * k] = make_float2(ldexpf(1.0f, E >> 1), ldexpf(1.0f, E - (E >> 1)));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] *= inv;
            const int slot = kscale_pos<BITS>(4 * lane + i);
            const int ln = 4 * (2 * warp) + ((slot >> 3) & 3);  // column 2 warp (hi), + 4 lanes: column 2 warp + 1 (lo)
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              const float x = part ? L * fmaxf(v[i], 0.0f) : v[i];
              const __half hi = __float2half_rn(x);
              reinterpret_cast<__half*>(&table[k][part][slot >> 5][ln])[slot & 7] = hi;
              reinterpret_cast<__half*>(&table[k][part][slot >> 5][ln + 4])[slot & 7] = __float2half_rn(x - __half2float(hi));
            }
          }
          if (cv.n_out > 0) *reinterpret_cast<float4*>(&qs[warp + 4 * k][4 * lane]) = make_float4(v[0], v[1], v[2], v[3]);
        }
        __syncthreads();
      }
#pragma unroll 1
      for (int k = 0; k < blocks; ++k) {
        float dz[4] = {0.f, 0.f, 0.f, 0.f}, ds[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 bz = table[k][0][c][lane], bs = table[k][1][c][lane];
          mma16816(dz, a[0][0][c].x, a[1][0][c].x, a[0][0][c].y, a[1][0][c].y, bz.x, bz.y);
          mma16816(ds, a[0][1][c].x, a[1][1][c].x, a[0][1][c].y, a[1][1][c].y, bs.x, bs.y);
          mma16816(dz, a[0][0][c].z, a[1][0][c].z, a[0][0][c].w, a[1][0][c].w, bz.z, bz.w);
          mma16816(ds, a[0][1][c].z, a[1][1][c].z, a[0][1][c].w, a[1][1][c].w, bs.z, bs.w);
        }
        // columns 2 tig, 2 tig + 1: head j0 + 4 k + tig, hi and lo
        float s0 = (dz[0] + ds[0]) + (dz[1] + ds[1]);
        float s1 = (dz[2] + ds[2]) + (dz[3] + ds[3]);
        if (cv.n_out > 0) {
          for (int r = 0; r < 16 && t0 + r < nb; ++r) {
            const uint8_t* ob = tiles + (long)(t0 + r) * cv.tile_bytes + kTileBytes<BITS>;
            const uint32_t iw = *reinterpret_cast<const uint32_t*>(ob);
            const __half* val = reinterpret_cast<const __half*>(ob + 16) + lane * cv.n_out;  // lane = token
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            for (int o = 0; o < cv.n_out; ++o) {
              const float x = __half2float(val[o]);
              const int ch = (iw >> (8 * o)) & 0xffu;
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] = fmaf(x, qs[4 * k + j][ch], v[j]);
            }
            float m = 0.0f;  // the largest over the tokens, for head tig
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float mj = warp_max(v[j]);
              m = tig == j ? mj : m;
            }
            if (g == (r & 7)) {
              if (r < 8) s0 += m;
              else s1 += m;
            }
          }
        }
        if (j0 + 4 * k + tig < grp) {
          const float2 p = qpow[4 * k + tig];
          best0 = fmaxf(best0, s0 * p.x * p.y);
          best1 = fmaxf(best1, s1 * p.x * p.y);
        }
      }
    }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
      best0 = fmaxf(best0, __shfl_xor_sync(kFull, best0, o));
      best1 = fmaxf(best1, __shfl_xor_sync(kFull, best1, o));
    }
    if (tig < 2) {
      const int t = t0 + g + 8 * tig;
      if (t < row) out[t] = t < nb ? (tig ? best1 : best0) : -INFINITY;
    }
  }
}

// ---------------------------------------------------------------------------
// Selection: one CTA per unit.  Scores map to integers of the same order (NaN
// below everything, -0 as +0).  The blocks that are always taken leave the
// contest; of the rest, the n-th largest key is found from histograms of eight
// bits at a time, beginning at the highest bit in which any two keys differ
// (scores of one unit share their leading bits, and would share one bin), and
// ending as soon as a whole bin is taken.  One ordered pass then writes the
// indices above the threshold and the first few equal to it.  Bound by the
// latency of its few barriers: up to K keys a thread stay in registers (K = 0:
// a row of any length is read again for every pass).  64 rows of 127 keys take
// 2.7 us, 8 rows of 4092 6.2 us, of which an empty launch is about 2; 1024
// threads of four keys for the latter (512 of eight: 6.8), 256 of four up to
// 1024 keys (beside an eviction 1.1 us less than 1024 threads).

__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The shared memory of a selection by NT threads.
template <int NT, int K>
struct SelectSmem {
  uint32_t hist[2][256];
  uint32_t min[NT / 32], max[NT / 32], cnt[(K > 0 ? K : 1) * NT / 32];
  uint32_t bin, above, in, total;
};

// The n chosen of a unit's nb blocks into out, ascending (the caller's barrier
// makes them visible).
template <int NT, int K>
__device__ __forceinline__ void select_unit(SelectSmem<NT, K>& sm, const float* sc, int nb, int n, int first, int last,
                                            int* out) {
  constexpr int NW = NT / 32, C = K > 0 ? K : 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lo = min(first, nb), hi = max(nb - last, lo);  // the contest
  int need = n - (nb - (hi - lo));                         // blocks it gives
  uint32_t key[C];
  if constexpr (K > 0) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int i = j * NT + tid;
      key[j] = i < nb ? order_key(sc[i]) : 0u;
    }
  }
  auto for_contest = [&](auto&& f) {
    if constexpr (K > 0) {
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const int i = j * NT + tid;
        if (i >= lo && i < hi) f(key[j]);
      }
    } else {
      for (int i = lo + tid; i < hi; i += NT) f(order_key(sc[i]));
    }
  };

  // taken of the contest: keys above `least`, and the first `need` equal to it
  uint32_t least = 0;
  const bool all = need >= hi - lo;
  if (!all && need > 0) {
    for (int i = tid; i < 256; i += NT) sm.hist[0][i] = 0;
    uint32_t mn = 0xffffffffu, mx = 0u;
    for_contest([&](uint32_t k) { mn = min(mn, k), mx = max(mx, k); });
    mn = __reduce_min_sync(kFull, mn);
    mx = __reduce_max_sync(kFull, mx);
    if (lane == 0) sm.min[warp] = mn, sm.max[warp] = mx;
    __syncthreads();
    mn = __reduce_min_sync(kFull, sm.min[lane % NW]);
    mx = __reduce_max_sync(kFull, sm.max[lane % NW]);
    int w = 32 - __clz((int)(mx - mn));  // undecided bits of key - mn (__clz(0) = 32)
    uint32_t prefix = 0;                 // its decided leading bits
    int cur = 0;
    bool whole = false;                  // the threshold's bin is taken whole
    while (w > 0 && !whole) {
      const int shift = max(w - 8, 0);
      const uint32_t digit = (1u << (w - shift)) - 1u;
      for_contest([&](uint32_t k) {
        const uint32_t r = k - mn;
        if ((w < 32 ? r >> w : 0u) == prefix) atomicAdd(&sm.hist[cur][(r >> shift) & digit], 1u);
      });
      __syncthreads();
      if (warp == 0) {
        // bins 8 lane .. 8 lane + 7; how many keys lie in the bins above them
        const uint4 x = reinterpret_cast<const uint4*>(sm.hist[cur])[2 * lane];
        const uint4 y = reinterpret_cast<const uint4*>(sm.hist[cur])[2 * lane + 1];
        const uint32_t c[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        uint32_t sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += c[i];
        uint32_t from = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_down_sync(kFull, from, o);
          if (lane + o < 32) from += v;
        }
        uint32_t above = from - sum;
        if (above < (uint32_t)need && from >= (uint32_t)need) {
          int bin = 8 * lane;
          uint32_t in = 0;
          bool found = false;
#pragma unroll
          for (int i = 7; i >= 0; --i) {
            if (found) continue;
            if (above + c[i] >= (uint32_t)need) {
              found = true, bin = 8 * lane + i, in = c[i];
            } else {
              above += c[i];
            }
          }
          sm.bin = (uint32_t)bin, sm.above = above, sm.in = in;
        }
      } else {
        for (int i = tid - 32; i < 256; i += NT - 32) sm.hist[cur ^ 1][i] = 0;
      }
      __syncthreads();
      need -= (int)sm.above;
      prefix = (w - shift < 32 ? prefix << (w - shift) : 0u) | sm.bin;
      whole = sm.in == (uint32_t)need;
      w = shift;
      cur ^= 1;
    }
    least = mn + (prefix << w);
    // every key from `least` on (above 0: some key of the contest stays out)
    if (whole) --least, need = 0;
  }

  // the ordered pass
  auto verdict = [&](int i, uint32_t k, bool& tie) {
    tie = false;
    if (i >= nb) return false;
    if (i < lo || i >= hi || all) return true;
    if (n - (nb - (hi - lo)) <= 0) return false;
    tie = k == least;
    return k > least;
  };
  int done = 0, ties = 0;  // taken above the threshold, equals, of the rounds before
  for (int i0 = 0; i0 < nb; i0 += C * NT) {
    uint32_t takes[C], equal[C];
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int i = i0 + j * NT + tid;
      bool tie;
      const bool take = verdict(i, K > 0 ? key[j] : (i < nb ? order_key(sc[i]) : 0u), tie);
      takes[j] = __ballot_sync(kFull, take);
      equal[j] = __ballot_sync(kFull, tie);
      if (lane == 0) sm.cnt[j * NW + warp] = __popc(takes[j]) | __popc(equal[j]) << 16;
    }
    __syncthreads();
    if (warp == 0) {  // exclusive sums over (round, warp)
      uint32_t run = 0;
      for (int e0 = 0; e0 < C * NW; e0 += 32) {
        const uint32_t v = e0 + lane < C * NW ? sm.cnt[e0 + lane] : 0u;
        uint32_t x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(kFull, x, o);
          if (lane >= o) x += y;
        }
        if (e0 + lane < C * NW) sm.cnt[e0 + lane] = run + x - v;
        run += __shfl_sync(kFull, x, 31);
      }
      if (lane == 0) sm.total = run;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const uint32_t before = sm.cnt[j * NW + warp], below = (1u << lane) - 1u;
      const int taken = done + (int)(before & 0xffffu) + __popc(takes[j] & below);
      const int rank = ties + (int)(before >> 16) + __popc(equal[j] & below);
      const int i = i0 + j * NT + tid;
      if (takes[j] >> lane & 1u) out[taken + min(rank, need)] = i;
      else if ((equal[j] >> lane & 1u) && rank < need) out[taken + rank] = i;
    }
    if (K == 0) {
      done += (int)(sm.total & 0xffffu);
      ties += (int)(sm.total >> 16);
      __syncthreads();  // the counts are read
    }
  }
}

// What stays of a unit's sums (SelectArgs::sums), by the CTA that has its list.
__device__ __forceinline__ void move_sums(const SelectArgs& a, long unit, int l, int nb, int n, const int* list) {
  const float* sc = a.scores + unit * a.row;
  // the sums of what stays: every read of a round is before its writes, and
  // a round reads nothing in front of itself (sources ascend, at or behind
  // their place), so `sums` may be `scores`
  const int held = (l + kGroup - 1) / kGroup - nb;  // the window's blocks
  float* to = a.sums + unit * a.sums_row;
  for (int i0 = 0; i0 < a.sums_row; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    float v = 0.0f;
    if (i < n) v = sc[list[i]];
    else if (i < n + held) v = sc[nb + i - n];
    __syncthreads();
    if (i < a.sums_row) to[i] = v;
  }
}

template <int NT, int K>
__global__ void __launch_bounds__(NT) select_kernel(CacheView cv, SelectArgs a, const SeqLens lens) {
  __shared__ __align__(16) SelectSmem<NT, K> sm;
  const int h = blockIdx.x, b = blockIdx.y;
  const long unit = (long)b * cv.H + h;
  const int l = seq_len(lens, b);
  const int nb = packed_blocks(l, cv.R, cv.policy);
  const int n = a.step > 0 ? evict_left(nb, a.n, a.step) : min(a.n, nb);
  int* out = a.out + unit * a.out_row;
  grid_dependency_wait();
  if (a.release) grid_launch_dependents();
  select_unit<NT, K>(sm, a.scores + unit * a.row, nb, n, a.first, a.last, out);
  for (int i = n + threadIdx.x; i < a.out_row; i += NT) out[i] = -1;
  if (a.sums == nullptr) return;
  __syncthreads();  // the list is written
  move_sums(a, unit, l, nb, n, out);
}

// ---------------------------------------------------------------------------
// Eviction: the tiles that stay, in order, at the front of their unit, and
// the window's tiles behind them.

// Source tile of place i: the i-th kept block, then the window's tiles.
__device__ __forceinline__ int evict_source(const int* kept, int left, int nb, int i) {
  return i < left ? kept[i] : nb + i - left;
}

// What moves in a sequence: its packed blocks, those that stay, and the
// places that they and the window's tiles take.
struct EvictPlan {
  int nb, left, places;
};
__device__ __forceinline__ EvictPlan evict_plan(const CacheView& cv, int l, int n_keep) {
  EvictPlan p;
  p.nb = packed_blocks(l, cv.R, cv.policy);
  p.left = evict_left(p.nb, n_keep, cv.W / kGroup);
  const int filled = (max(policy_nq_k(l, cv.R, cv.policy), policy_nq_v(l, cv.R, cv.policy)) + kGroup - 1) / kGroup;
  p.places = p.left + filled - p.nb;
  return p;
}

// n 16-byte words by the lanes of a warp, kFlight of a lane in flight.
constexpr int kFlight = 6;
__device__ __forceinline__ void warp_copy(uint4* d, const uint4* s, long n, int lane) {
  for (long w0 = lane; w0 < n; w0 += 32 * kFlight) {
    uint4 v[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
      if (w0 + 32 * k < n) v[k] = __ldcs(s + w0 + 32 * k);
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
      if (w0 + 32 * k < n) __stcs(d + w0 + 32 * k, v[k]);
  }
}

// Into another cache: a warp per place, and past the places a warp per ring.
// 64 units of 256 kept 5 KB tiles and their rings: 24 us for the 174 MB read
// and written, the rate of a plain copy (34 us with the selection before it).
constexpr int kEvictWarps = 4;
__global__ void __launch_bounds__(32 * kEvictWarps)
    evict_copy_kernel(CacheView src, CacheView dst, const int* kept, int kept_row, int n_keep, int most,
                      const SeqLens lens) {
  const int h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31;
  const int i = blockIdx.x * kEvictWarps + (threadIdx.x >> 5);
  const long unit = (long)b * src.H + h;
  grid_dependency_wait();  // the list, and whatever came before it
  if (i >= most) {
    const long row = (long)src.W * kHeadDim / 8;
    if (i == most) warp_copy(reinterpret_cast<uint4*>(dst.ring_k) + unit * row, reinterpret_cast<const uint4*>(src.ring_k) + unit * row, row, lane);
    if (i == most + 1) warp_copy(reinterpret_cast<uint4*>(dst.ring_v) + unit * row, reinterpret_cast<const uint4*>(src.ring_v) + unit * row, row, lane);
    return;
  }
  const EvictPlan p = evict_plan(src, seq_len(lens, b), n_keep);
  if (i >= p.places) return;
  const long from = unit * (src.Tcap / kGroup) + evict_source(kept + unit * kept_row, p.left, p.nb, i);
  const long to = unit * (dst.Tcap / kGroup) + i;
  warp_copy(reinterpret_cast<uint4*>(dst.tiles + to * dst.tile_bytes),
            reinterpret_cast<const uint4*>(src.tiles + from * src.tile_bytes), src.tile_bytes / 16, lane);
}

// Rows of up to kEvictRow blocks, into another cache, in one launch: every CTA
// of a unit makes the choice again (about 1 us, for the 2 us of a launch); its
// first one writes the list and the sums.  64 units of 127 blocks, 33 kept: 6.3
// us, 7.0 as two launches; rows of 1022 blocks would take 38.6 us for 34.
constexpr int kEvictRow = 512;
__global__ void __launch_bounds__(32 * kEvictWarps)
    evict_small_kernel(CacheView src, CacheView dst, SelectArgs a, int most, const SeqLens lens) {
  __shared__ __align__(16) SelectSmem<32 * kEvictWarps, kEvictRow / (32 * kEvictWarps)> sm;
  __shared__ int list[kEvictRow];
  const int h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31;
  const int i = blockIdx.x * kEvictWarps + (threadIdx.x >> 5);
  const long unit = (long)b * src.H + h;
  const int l = seq_len(lens, b);
  const EvictPlan p = evict_plan(src, l, a.n);
  grid_dependency_wait();
  if (i >= most) {
    const long row = (long)src.W * kHeadDim / 8;
    if (i == most) warp_copy(reinterpret_cast<uint4*>(dst.ring_k) + unit * row, reinterpret_cast<const uint4*>(src.ring_k) + unit * row, row, lane);
    if (i == most + 1) warp_copy(reinterpret_cast<uint4*>(dst.ring_v) + unit * row, reinterpret_cast<const uint4*>(src.ring_v) + unit * row, row, lane);
  }
  if ((int)blockIdx.x * kEvictWarps >= max(p.places, 1)) return;  // (the first CTA writes its row all the same)
  select_unit<32 * kEvictWarps, kEvictRow / (32 * kEvictWarps)>(sm, a.scores + unit * a.row, p.nb, p.left, a.first,
                                                               a.last, list);
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int k = threadIdx.x; k < a.out_row; k += blockDim.x) a.out[unit * a.out_row + k] = k < p.left ? list[k] : -1;
    if (a.sums != nullptr) move_sums(a, unit, l, p.nb, p.left, list);
  }
  if (i >= min(p.places, most)) return;
  const long from = unit * (src.Tcap / kGroup) + evict_source(list, p.left, p.nb, i);
  const long to = unit * (dst.Tcap / kGroup) + i;
  warp_copy(reinterpret_cast<uint4*>(dst.tiles + to * dst.tile_bytes),
            reinterpret_cast<const uint4*>(src.tiles + from * src.tile_bytes), src.tile_bytes / 16, lane);
}

// In place: a thread owns one 16-byte column of a unit's tiles and walks the
// places in order.  A source never lies in front of its place, so a thread
// reads what it has not yet written, and no other thread touches its column;
// kAhead reads go out before their writes.  The rings stay.
__global__ void __launch_bounds__(64)
    evict_inplace_kernel(CacheView cv, const int* kept, int kept_row, int n_keep, const SeqLens lens) {
  const int h = blockIdx.y, b = blockIdx.z;
  const long unit = (long)b * cv.H + h;
  grid_dependency_wait();
  const EvictPlan p = evict_plan(cv, seq_len(lens, b), n_keep);
  const int col = blockIdx.x * blockDim.x + threadIdx.x;
  if (col * 16 >= cv.tile_bytes || p.left == p.nb) return;
  uint8_t* base = cv.tiles + unit * (cv.Tcap / kGroup) * (long)cv.tile_bytes + 16 * col;
  const int* list = kept + unit * kept_row;
  constexpr int kAhead = 16;
  for (int i0 = 0; i0 < p.places; i0 += kAhead) {
    uint4 v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i0 + k < p.places)
        v[k] = *reinterpret_cast<const uint4*>(base + (long)evict_source(list, p.left, p.nb, i0 + k) * cv.tile_bytes);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i0 + k < p.places) *reinterpret_cast<uint4*>(base + (long)(i0 + k) * cv.tile_bytes) = v[k];
  }
}

// ---------------------------------------------------------------------------
// Block weights: with (M, T) the softmax's max and sum of a head over all
// tokens and (m, t) those of a block, the block's weight is the sum over the
// unit's heads of t 2^(m - M) / T.  A thread takes a block and sums its heads
// in order.  About 3 us behind an attention of 131k tokens; short rows are
// taken by the attention itself (fold_mass).
constexpr int kMassThreads = 128;

__global__ void __launch_bounds__(kMassThreads) mass_kernel(CacheView cv, MassArgs a, const SeqLens lens) {
  const int h = blockIdx.y, b = blockIdx.z;
  const long unit = (long)b * cv.H + h;
  const int blocks = (seq_len(lens, b) + kGroup - 1) / kGroup;
  const int grp = a.Hq / cv.H, nhc = (grp + kHeadChunk - 1) / kHeadChunk;
  const int i = blockIdx.x * kMassThreads + threadIdx.x;
  grid_dependency_wait();
  if (i >= a.row) return;
  const float before = a.mass_in ? a.decay * a.mass_in[unit * a.row + i] : 0.0f;
  float w = 0.0f;
  if (i < blocks) {
    for (int hc = 0; hc < nhc; ++hc) {
      const int nh = min(kHeadChunk, grp - hc * kHeadChunk);
      const long gid = unit * nhc + hc;
      // two heads a load, the loads of four heads at once
      const float4* rec = reinterpret_cast<const float4*>(a.records + (gid * a.record_blocks + i) * kHeadChunk);
      const float4* all = reinterpret_cast<const float4*>(a.totals + gid * kHeadChunk);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (4 * half >= nh) break;
        const float4 r[2] = {rec[2 * half], rec[2 * half + 1]}, t[2] = {all[2 * half], all[2 * half + 1]};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int j = 4 * half + 2 * k;
          if (j < nh) w += r[k].y * fast_exp2(r[k].x - t[k].x) / t[k].y;
          if (j + 1 < nh) w += r[k].w * fast_exp2(r[k].z - t[k].z) / t[k].w;
        }
      }
    }
  }
  a.mass_out[unit * a.row + i] = before + w;
}

}  // namespace

// Every launch here may start as the one before it on the stream ends; it
// waits for it (grid_dependency_wait) before it touches memory.  It lets the
// next one start at its exit, or, where `release` says that the next one is
// another kernel of the same call (which waits too), right after its own wait:
// an attention call with the overlap on reads its q and its cache without
// waiting, and the last launch of any other call has to be complete by then.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t st, A... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(threads);
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, args...);
}

cudaError_t launch_block_scores(const CacheView& cv, const void* q, int q_dtype, int Hq, float* scores, int row,
                                bool release, const SeqLens& lens, cudaStream_t st) {
  // four CTAs an SM (their loads in flight are 128 KB): one wave, or a CTA a unit
  const long wave = 4l * kTargetSMs / ((long)cv.H * cv.B);
  const int need = (row + kScoreTiles - 1) / kScoreTiles;
  const dim3 grid(need < wave ? need : (wave > 1 ? (int)wave : 1), cv.H, cv.B);
  auto kernel = score_kernel<8>;
  if (cv.bits == 2) kernel = score_kernel<2>;
  if (cv.bits == 3) kernel = score_kernel<3>;
  if (cv.bits == 4) kernel = score_kernel<4>;
  const int wide = ((uintptr_t)q & 15u) == 0;
  return launch_early(kernel, grid, 32 * kScoreWarps, st, cv, q, q_dtype, wide, Hq / cv.H, scores, row, (int)release,
                      lens);
}

cudaError_t launch_select(const CacheView& cv, const SelectArgs& a, int most, const SeqLens& lens, cudaStream_t st) {
  const dim3 grid(cv.H, cv.B);
  if (most <= 512) return launch_early(select_kernel<128, 4>, grid, 128, st, cv, a, lens);
  if (most <= 1024) return launch_early(select_kernel<256, 4>, grid, 256, st, cv, a, lens);
  if (most <= 4096) return launch_early(select_kernel<1024, 4>, grid, 1024, st, cv, a, lens);
  return launch_early(select_kernel<1024, 0>, grid, 1024, st, cv, a, lens);
}

cudaError_t launch_evict(const CacheView& src, const CacheView& dst, const SelectArgs& a, int blocks, int most,
                         const SeqLens& lens, cudaStream_t st) {
  const int* kept = a.out;
  const int kept_row = a.out_row, n_keep = a.n;
  // (sums that take the scores' own memory wait for every CTA's choice)
  const bool apart = a.sums == nullptr || a.sums >= a.scores + (long)src.B * src.H * a.row ||
                     a.scores >= a.sums + (long)src.B * src.H * a.sums_row;
  if (src.tiles != dst.tiles && blocks <= kEvictRow && apart) {
    const dim3 grid((most + 2 + kEvictWarps - 1) / kEvictWarps, src.H, src.B);
    return launch_early(evict_small_kernel, grid, 32 * kEvictWarps, st, src, dst, a, most, lens);
  }
  const cudaError_t e = launch_select(src, a, blocks, lens, st);
  if (e != cudaSuccess) return e;
  if (src.tiles == dst.tiles) {
    const dim3 grid((src.tile_bytes / 16 + 63) / 64, src.H, src.B);
    return launch_early(evict_inplace_kernel, grid, 64, st, src, kept, kept_row, n_keep, lens);
  }
  const dim3 grid((most + 2 + kEvictWarps - 1) / kEvictWarps, src.H, src.B);
  return launch_early(evict_copy_kernel, grid, 32 * kEvictWarps, st, src, dst, kept, kept_row, n_keep, most, lens);
}

cudaError_t launch_mass(const CacheView& cv, const MassArgs& a, const SeqLens& lens, cudaStream_t st) {
  const dim3 grid((a.row + kMassThreads - 1) / kMassThreads, cv.H, cv.B);
  return launch_early(mass_kernel, grid, kMassThreads, st, cv, a, lens);
}

}  // namespace kivi
