// Backward of sliding-window attention with sinks for gfx950.
//
//   p_tj = exp(scale q_t.k_j - lse_t), dp_tj = dy_t.v_j
//   ds_tj = p_tj (dp_tj - dy_t.y_t)
//   dq_t = scale sum_j ds_tj k_j, dk_j = scale sum_t ds_tj q_t, dv_j = sum_t p_tj dy_t
//
// Two kernels, so that every sum has one owner and no atomics: one walks the
// keys of 32 queries per wavefront (dq), the other the queries and heads of 32
// keys per wavefront (dk, dv).  That is 7 products of pairs x headdim, 8 with
// the second part of ds below, against the 5 that a single pass would need,
// which would have to add dq from many workgroups.  p and ds go from one
// product's result into the next one's operand as they lie (see swa_tile.h);
// everything is summed in float32.
//
// Roundings.  The matrix cores take p and ds in bfloat16.  For dk and dv they
// are rounded: the error is 2.3e-3 of their norm, where rounding the results
// alone gives 1.65e-3; a second part of both would give that, and take a
// quarter to two fifths more time (8192 tokens, 16 heads of 128, window 1024:
// 223 -> 281 us; 4 x 4096 tokens over all their past, 32 heads of 64: 691 -> 918).
// dq would also have the error of dy.y, which comes from the rounded y and in
// rows of few keys weighs as much as a rounding of dq: 2.6e-3.  So ds goes into
// dq in two parts, rounded and left over (1.8e-3 to 2.1e-3, for 15 to 24% of
// the kernel: 130 -> 157 us and 501 -> 620 in those cases, 66 -> 76 on 4 ragged
// rows of 2048, window 512).  dq keeps the inexact dy.y, but the sum of ds tells
// what it lacks, and dk takes the exact one.
//
// Bound as the forward is (matrix instructions busy a third of the time): dq and
// dk with dv of 8192 tokens, 16 heads of 128 on 4, window 1024, 157 and 223 us
// (820 and 580 TFLOP/s of what they compute); 4 x 2048 tokens, 32 heads of 64 on
// 8, window 512, 100 and 110 us (600 and 550).
#include <type_traits>

#include "swa_tile.h"

namespace ssmb {
namespace {

// What a workgroup of the dq kernel knows of its work, and a lane of its query.
struct DqWork {
  const uint16_t *k, *v;  // of the key head
  int q0, wq0, len, tiles;
  KeyRow keys;
  float c2, lse2, delta;
};

// One pass over the keys: dq of the lane's query, and off, what dy.y is too
// small by, since y is rounded: the weights' sum is 1, so sum_j ds_tj (of this
// lane's half of the keys).  Returns whether a tile that some query sees in
// part had a score that is not finite.  An infinity or NaN in a key makes every
// score with it one, and 0 times it would reach the queries that do not see it:
// SAFE keeps such elements out of the product, and gives a NaN to the queries
// that do (whose ds is NaN or 0 there).
template <int D, bool SAFE>
__device__ __forceinline__ bool dq_pass(const SwaParams &p, const DqWork &w, u4 (&lds)[2][2][kTile * D / 8],
                                        const bf8 (&q)[D / 16], const bf8 (&dy)[D / 16], f16v (&dq)[D / 32], float &off,
                                        int tid) {
  constexpr int NB = D / 32, NS = D / 16;
  const int lane = tid & 63, half = lane >> 5, t = w.wq0 + (lane & 31);
  const int window = static_cast<int>(p.window), sinks = static_cast<int>(p.sinks);
  const Lanes at = lanes_of<D>(lane);
  float even = 0.0f;  // NaN once a score was not finite
  off = 0.0f;
#pragma unroll
  for (int db = 0; db < NB; ++db) dq[db] = f16v{};
  auto start = [&](int i) {
    load_keys<D, 256>(lds[i & 1][0], w.k, p.k_token, w.keys, i * kTile, w.len - 1, tid);
    load_keys<D, 256>(lds[i & 1][1], w.v, p.v_token, w.keys, i * kTile, w.len - 1, tid);
  };
  start(0);
  for (int i = 0; i < w.tiles; ++i) {
    wait_tiles();
    __syncthreads();  // tile i has landed, and nobody reads the other buffer any more
    if (i + 1 < w.tiles) start(i + 1);
    const int v0 = i * kTile, j0 = w.keys.key(v0), j1 = w.keys.key(v0 + kTile - 1);
    const u4 *kt = lds[i & 1][0], *vt = lds[i & 1][1];
    if (j0 > w.wq0 + 31 || (j1 <= w.wq0 - window && j0 >= sinks) || w.wq0 >= w.len) continue;
    const bool whole = j1 <= w.wq0 && w.wq0 + 31 - j0 < window;
    const Seen seen = seen_by(w.keys, t, v0, half, window, sinks);
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      f16v s = {}, dp = {};
#pragma unroll
      for (int ks = 0; ks < NS; ++ks) {
        s = mfma(row_operand<D>(kt, 32 * blk, ks, at), q[ks], s);
        dp = mfma(row_operand<D>(vt, 32 * blk, ks, at), dy[ks], dp);
      }
      reads_ahead<2 * NS>();
#pragma unroll
      for (int r = 0; r < 16; ++r)
        dp[r] = __builtin_amdgcn_exp2f(fmaf(s[r], w.c2, -w.lse2)) * (dp[r] - w.delta);
      if (!whole) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          if constexpr (!SAFE) even = fmaf(s[r], 0.0f, even);
          dp[r] = seen(32 * blk + d_row(r, 0)) ? dp[r] : 0.0f;
        }
        if constexpr (SAFE) {
          bf8 vis[2];
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int e = 0; e < 8; ++e) vis[ks][e] = static_cast<__bf16>(seen(32 * blk + d_row(8 * ks + e, 0)) ? 1.0f : 0.0f);
          add_not_finite<D, 2, true>(kt, 32 * blk, vis, dq, at);
        }
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) off += dp[r];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const bf8 dsk = as_operand(dp, ks), rest = left_over(dp, ks, dsk);
#pragma unroll
        for (int db = 0; db < NB; ++db) {
          bf8 kc = col_operand<D>(kt, 32 * blk + 16 * ks, db, at);
          if constexpr (SAFE) {
            if (!whole) kc = only_finite(kc);
          }
          dq[db] = mfma(kc, dsk, dq[db]);
          dq[db] = mfma(kc, rest, dq[db]);
          if constexpr (SAFE) __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }
  return even != 0.0f;
}

// dq; also log2(e) lse and dy.y of every query for the kernel below.  Three
// workgroups per CU with headdim 64 (what does not fit its registers is in the
// rare pass).
template <int D>
__global__ void __launch_bounds__(256, D == 64 ? 3 : 2) swa_dq_kernel(const SwaParams p, int hw, unsigned qtiles, unsigned n) {
  constexpr int CH = D / 8, NB = D / 32, NS = D / 16;
  __shared__ __align__(16) u4 lds[2][2][kTile * CH];  // buffer, K or V
  __shared__ int found;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const unsigned nheads = static_cast<unsigned>(p.nheads), nkv = static_cast<unsigned>(p.nkv);
  const unsigned group = nheads / nkv, hb = group / hw;
  const unsigned batch = static_cast<unsigned>(p.batch), id = xcd_order(blockIdx.x, n, nkv * batch);
  const unsigned rest = id / qtiles, qt = uneven(p.window, p.seqlen) ? qtiles - 1 - id % qtiles : id % qtiles;
  const int64_t c = rest / (hb * batch), b = rest / hb % batch;
  const int64_t head = c * group + (rest % hb) * hw + wave % hw;
  const int qspan = 32 * (4 / hw), q0 = static_cast<int>(qt) * qspan;
  DqWork w;
  w.q0 = q0;
  w.wq0 = q0 + 32 * (wave / hw);
  w.len = row_length(p, b);
  const int last = w.len - 1, t = w.wq0 + (lane & 31), L = static_cast<int>(p.seqlen);
  const int64_t out = ((b * p.seqlen + t) * p.nheads + head) * D;

  f16v dq[NB] = {};
  if (q0 < w.len) {
    const int qlast = q0 + qspan - 1 < last ? q0 + qspan - 1 : last;
    w.keys = key_row(q0, static_cast<int>(p.window), static_cast<int>(p.sinks));
    w.tiles = (w.keys.first + qlast - w.keys.low) / kTile + 1;
    w.k = p.k + b * p.k_batch + c * D;
    w.v = p.v + b * p.v_batch + c * D;
    bf8 q[NS], dy[NS];
    const int row = t < last ? t : last;
    const int64_t from = ((b * p.seqlen + row) * p.nheads + head) * D;
    const u4 *qs = reinterpret_cast<const u4 *>(p.q + b * p.q_batch + row * p.q_token + head * D);
    const u4 *ds = reinterpret_cast<const u4 *>(p.dy + from), *ys = reinterpret_cast<const u4 *>(p.y + from);
    float delta = 0.0f, off;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      q[s] = __builtin_bit_cast(bf8, qs[2 * s + half]);
      dy[s] = __builtin_bit_cast(bf8, ds[2 * s + half]);
      const u4 d4 = ds[2 * s + half], y4 = ys[2 * s + half];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        delta = fmaf(__uint_as_float(d4[e] << 16), __uint_as_float(y4[e] << 16), delta);
        delta = fmaf(__uint_as_float(d4[e] & 0xffff0000u), __uint_as_float(y4[e] & 0xffff0000u), delta);
      }
    }
    w.delta = delta + other_half(delta);
    const int64_t stat = (b * p.nheads + head) * p.seqlen + row;
    w.lse2 = p.lse[stat] * kLog2e;
    w.c2 = p.scale * kLog2e;
    if (tid == 0) found = 0;  // before the first barrier in dq_pass()
    const bool bad = dq_pass<D, false>(p, w, lds, q, dy, dq, off, tid);
    if (__any(bad)) found = 1;
    __syncthreads();
    if (found) dq_pass<D, true>(p, w, lds, q, dy, dq, off, tid);
    off += other_half(off);
    if (half == 0 && t < w.len) {
      p.ws_lse2[stat] = w.lse2;
      p.ws_delta[stat] = w.delta + off;
    }
  }
  if (t >= L) return;
#pragma unroll
  for (int db = 0; db < NB; ++db)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf4 v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = static_cast<__bf16>(t < w.len ? dq[db][4 * j + r] * p.scale : 0.0f);
      *reinterpret_cast<bf4 *>(p.dq + out + 32 * db + 8 * j + 4 * half) = v;
    }
}

// The gradients that 32 queries (rows base .. base + 31 of the tiles qt and dt,
// with their stats) give the 32 keys of a wavefront, lane % 32 its key.  WHOLE:
// every query sees every key; else sees(row) tells, rows less 4 in the second lane half.
//
// An infinity or NaN in a query or its dy, times 0, would reach the keys that it
// does not see: SAFE keeps such elements out of the products and adds what they
// are worth (dv: p is above 0; dk: ds is NaN or 0) to the keys that it sees.
template <int D, bool SAFE, typename F>
__device__ __forceinline__ void add_queries(const u4 *qt, const u4 *dt, const float *lse2, const float *delta, int base,
                                            const bf8 (&kf)[D / 16], const bf8 (&vf)[D / 16], float c2, bool whole, F sees,
                                            f16v (&dk)[D / 32], f16v (&dv)[D / 32], const Lanes &at, int half) {
  constexpr int NB = D / 32, NS = D / 16;
  f16v s = {}, dp = {};
#pragma unroll
  for (int ks = 0; ks < NS; ++ks) {
    s = mfma(row_operand<D>(qt, base, ks, at), kf[ks], s);
    dp = mfma(row_operand<D>(dt, base, ks, at), vf[ks], dp);
  }
  reads_ahead<2 * NS>();
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const float4 l4 = *reinterpret_cast<const float4 *>(lse2 + base + 8 * g + 4 * half);
    const float4 d4 = *reinterpret_cast<const float4 *>(delta + base + 8 * g + 4 * half);
    const float l[4] = {l4.x, l4.y, l4.z, l4.w}, d[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      s[4 * g + r] = __builtin_amdgcn_exp2f(fmaf(s[4 * g + r], c2, -l[r]));
      dp[4 * g + r] = s[4 * g + r] * (dp[4 * g + r] - d[r]);
    }
  }
  if (!whole) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const bool yes = sees(d_row(r, 0));
      s[r] = yes ? s[r] : 0.0f;
      dp[r] = yes ? dp[r] : 0.0f;
    }
    if constexpr (SAFE) {
      bf8 vis[2];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int e = 0; e < 8; ++e) vis[ks][e] = static_cast<__bf16>(sees(d_row(8 * ks + e, 0)) ? 1.0f : 0.0f);
      add_not_finite<D, 2, false>(dt, base, vis, dv, at);
      add_not_finite<D, 2, true>(qt, base, vis, dk, at);
    }
  }
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    const bf8 pk = as_operand(s, ks), dsk = as_operand(dp, ks);
#pragma unroll
    for (int db = 0; db < NB; ++db) {
      bf8 dc = col_operand<D>(dt, base + 16 * ks, db, at), qc = col_operand<D>(qt, base + 16 * ks, db, at);
      if constexpr (SAFE) {
        if (!whole) {
          dc = only_finite(dc);
          qc = only_finite(qc);
        }
      }
      dv[db] = mfma(dc, pk, dv[db]);
      dk[db] = mfma(qc, dsk, dk[db]);
      if constexpr (SAFE) __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// The keys and values of a wavefront as B operands.
template <int D>
__device__ __forceinline__ void load_keys_and_values(const SwaParams &p, int64_t b, int64_t c, int row, int half,
                                                     bf8 (&kf)[D / 16], bf8 (&vf)[D / 16]) {
  const u4 *ks = reinterpret_cast<const u4 *>(p.k + b * p.k_batch + row * p.k_token + c * D);
  const u4 *vs = reinterpret_cast<const u4 *>(p.v + b * p.v_batch + row * p.v_token + c * D);
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    kf[s] = __builtin_bit_cast(bf8, ks[2 * s + half]);
    vf[s] = __builtin_bit_cast(bf8, vs[2 * s + half]);
  }
}

// A D result, elements of 32 keys, as rows of D floats.
template <int D>
__device__ __forceinline__ void put_rows(float *to, int row, int half, const f16v (&v)[D / 32]) {
#pragma unroll
  for (int db = 0; db < D / 32; ++db)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<float4 *>(to + row * D + 32 * db + 8 * g + 4 * half) =
          make_float4(v[db][4 * g], v[db][4 * g + 1], v[db][4 * g + 2], v[db][4 * g + 3]);
}

__device__ __forceinline__ void add(float4 &a, const float4 &x) {
  a.x += x.x;
  a.y += x.y;
  a.z += x.z;
  a.w += x.w;
}

// The first query tile past those that see a block of 128 keys through the window.
__device__ __forceinline__ int far_tile(int b0, int window, int len) {
  const int reach = len - b0 <= window + 127 ? len : b0 + 127 + window;
  return (reach + kTile - 1) / kTile;
}

// dk and dv of 128 keys, 32 per wavefront, over the queries that see them
// through the window, or of the sinks among 32 keys over the queries past it
// (see SwaBwdPlan).  Two workgroups per CU with headdim 64; with 128 the sums
// and operands need more than half the registers, and one per CU that has them
// all took 567 us against 673 for two that spill (2 x 4096 tokens, 32 heads on
// 8, window 1024).
template <int D>
__global__ void __launch_bounds__(256, D == 64 ? 2 : 1) swa_dkv_kernel(const SwaParams p, const SwaBwdPlan plan, unsigned n) {
  constexpr int CH = D / 8, NB = D / 32, NS = D / 16;
  __shared__ __align__(16) u4 lds[2][2][kTile * CH];  // buffer, Q or dy
  __shared__ __align__(16) float stats[4][2][kTile];  // buffer or wavefront, log2(e) lse or dy.y
  __shared__ int found;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const unsigned nkv = static_cast<unsigned>(p.nkv), group = static_cast<unsigned>(p.nheads) / nkv;
  // The far items come last, where they fill what the others leave.
  const unsigned far_items = plan.far_blocks * plan.far_chunks, near_items = plan.blocks * plan.slices;
  const unsigned nnear = n / (far_items + near_items) * near_items;
  const bool far = blockIdx.x >= nnear;
  const unsigned batch = static_cast<unsigned>(p.batch);
  const unsigned item = far ? xcd_order(blockIdx.x - nnear, n - nnear, nkv * batch) : xcd_order(blockIdx.x, nnear, nkv * batch);
  const unsigned per = far ? far_items : near_items, k = item % per;
  const int64_t c = item / per / batch, b = item / per % batch, bc = b * nkv + c;
  const int len = row_length(p, b), last = len - 1, L = static_cast<int>(p.seqlen);
  const int window = static_cast<int>(p.window), sinks = static_cast<int>(p.sinks);
  const float c2 = p.scale * kLog2e;
  const Lanes at = lanes_of<D>(lane);
  f16v dk[NB] = {}, dv[NB] = {};
  bf8 kf[NS], vf[NS];
  // An infinity or NaN in a query makes its lse one, or -infinity, and one in its
  // dy makes dy.y one; NaN once such a query was met: then all over, safely.
  float even = 0.0f;

  if (far) {
    // Each wavefront walks (query tile of 32, head) pairs of its own, in LDS of its own.
    const unsigned fb = k / plan.far_chunks, chunk = k % plan.far_chunks;
    const int j0 = static_cast<int>(fb) * 32, j = j0 + (lane & 31);
    const int first = 2 * far_tile(j0 / 128 * 128, window, len), tiles = (len + 31) / 32 - first;
    const int units = tiles > 0 ? tiles * static_cast<int>(group) : 0, step = 4 * static_cast<int>(plan.far_chunks);
    u4 *qt = &lds[0][0][0] + wave * (2 * 32 * CH), *dt = qt + 32 * CH;
    if (units > 0) load_keys_and_values<D>(p, b, c, j < last ? j : last, half, kf, vf);
    auto start = [&](int u) {
      const int t0 = (first + u % tiles) * 32, head = static_cast<int>(c * group) + u / tiles;
      load_tile<D, 64, 32>(qt, p.q + b * p.q_batch + head * D, p.q_token, t0, last, lane);
      load_tile<D, 64, 32>(dt, p.dy + (b * p.seqlen * p.nheads + head) * D, p.nheads * D, t0, last, lane);
      load_stats(stats[wave][0], p.ws_lse2 + (b * p.nheads + head) * p.seqlen, t0, last, lane);
      load_stats(stats[wave][1], p.ws_delta + (b * p.nheads + head) * p.seqlen, t0, last, lane);
    };
    auto pass = [&](auto safe) {
      for (int u = static_cast<int>(chunk) * 4 + wave; u < units; u += step) {
        start(u);
        wait_tiles();
        const float look = stats[wave][half][lane & 31];
        const int t0 = (first + u % tiles) * 32;
        add_queries<D, decltype(safe)::value>(
            qt, dt, stats[wave][0], stats[wave][1], 0, kf, vf, c2, t0 + 31 < len && j0 + 31 < sinks,
            [&](int r) { return t0 + 4 * half + r < len && j < sinks; }, dk, dv, at, half);
        even = fmaf(look, 0.0f, even);
        wait_reads();
      }
    };
    pass(std::false_type());
    if (__any(even != 0.0f)) {
#pragma unroll
      for (int db = 0; db < NB; ++db) dk[db] = dv[db] = f16v{};
      pass(std::true_type());
    }
    // Add the wavefronts' terms, dk then dv, in LDS.
    float *sums = reinterpret_cast<float *>(lds), *out = p.ws_far + (bc * far_items + k) * 2 * 32 * D;
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
      put_rows<D>(sums + wave * 32 * D, lane & 31, half, which == 0 ? dk : dv);
      __syncthreads();
      for (int i = tid * 4; i < 32 * D; i += 1024) {
        float4 a = *reinterpret_cast<const float4 *>(sums + i);
#pragma unroll
        for (int w = 1; w < 4; ++w) add(a, *reinterpret_cast<const float4 *>(sums + w * 32 * D + i));
        *reinterpret_cast<float4 *>(out + which * 32 * D + i) = a;
      }
    }
    return;
  }

  const unsigned slice = k % plan.slices, block = k / plan.slices;
  const int heads = group / plan.slices, head0 = static_cast<int>(c * group + slice * heads);
  const int b0 = static_cast<int>(block) * 128, wk0 = b0 + 32 * wave, j = wk0 + (lane & 31);  // j: this lane's key
  // Query tiles: from the block's own to the last that sees one of its keys
  // (of the sinks, without far items: to the end).
  const int t_lo = b0 / kTile;
  const int t_hi = b0 >= len ? 0 : b0 < sinks && far_items == 0 ? (len + kTile - 1) / kTile : far_tile(b0, window, len);
  const int nq = t_hi > t_lo ? t_hi - t_lo : 0, steps = nq * heads;
  if (steps > 0) {
    load_keys_and_values<D>(p, b, c, j < last ? j : last, half, kf, vf);
    // How many queries from its own on see this lane's key: the window's, or all of a sink's, up to the length.
    const unsigned reach = j >= len ? 0 : j < sinks || window > len - j ? len - j : window;
    auto pass = [&](auto safe) {
      int at_head = head0, at_tile = t_lo;  // of the next tile to start
      auto start = [&](int i) {
        const int t0 = at_tile * kTile, buf = i & 1;
        load_tile<D, 256>(lds[buf][0], p.q + b * p.q_batch + at_head * D, p.q_token, t0, last, tid);
        load_tile<D, 256>(lds[buf][1], p.dy + (b * p.seqlen * p.nheads + at_head) * D, p.nheads * D, t0, last, tid);
        if (wave < 2) load_stats(stats[buf][wave], (wave == 0 ? p.ws_lse2 : p.ws_delta) + (b * p.nheads + at_head) * p.seqlen,
                                 t0, last, lane);
        if (++at_tile == t_hi) {
          at_tile = t_lo;
          ++at_head;
        }
      };
      start(0);
      int tile = t_lo;
      for (int i = 0; i < steps; ++i) {
        wait_tiles();
        __syncthreads();
        if (i + 1 < steps) start(i + 1);
        const float look = stats[i & 1][lane >> 4 & 1][16 * wave + (lane & 15)];  // a quarter of the queries
        const int t0 = tile * kTile;
        if (++tile == t_hi) tile = t_lo;
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          const int q0 = t0 + 32 * blk;
          // Does any of these 32 queries see any of the wavefront's keys, or all of them all?
          if (q0 + 31 < wk0 || (q0 >= wk0 + 31 + window && wk0 >= sinks) || q0 >= len || wk0 >= len) continue;
          const bool whole = q0 >= wk0 + 31 && q0 + 31 < len && (q0 + 31 - wk0 < window || wk0 + 31 < sinks);
          const int behind = q0 + 4 * half - j;  // of the lane's first query after its key
          add_queries<D, decltype(safe)::value>(
              lds[i & 1][0], lds[i & 1][1], stats[i & 1][0], stats[i & 1][1], 32 * blk, kf, vf, c2, whole,
              [&](int r) { return static_cast<unsigned>(behind + r) < reach; }, dk, dv, at, half);
        }
        even = fmaf(look, 0.0f, even);
      }
    };
    if (tid == 0) found = 0;  // before the first barrier in pass()
    pass(std::false_type());
    if (__any(even != 0.0f)) found = 1;
    __syncthreads();
    if (found) {
#pragma unroll
      for (int db = 0; db < NB; ++db) dk[db] = dv[db] = f16v{};
      pass(std::true_type());
    }
  }
  if (block < plan.sum_blocks) {
    const int64_t part = (bc * plan.sum_blocks + block) * plan.slices + slice;
    put_rows<D>(p.ws_part + part * 2 * 128 * D, 32 * wave + (lane & 31), half, dk);
    put_rows<D>(p.ws_part + (part * 2 + 1) * 128 * D, 32 * wave + (lane & 31), half, dv);
    return;
  }
  if (j >= L) return;
  const int64_t out = ((b * p.seqlen + j) * p.nkv + c) * D;
#pragma unroll
  for (int db = 0; db < NB; ++db)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      bf4 a, v;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        a[r] = static_cast<__bf16>(j < len ? dk[db][4 * g + r] * p.scale : 0.0f);
        v[r] = static_cast<__bf16>(j < len ? dv[db][4 * g + r] : 0.0f);
      }
      *reinterpret_cast<bf4 *>(p.dk + out + 32 * db + 8 * g + 4 * half) = a;
      *reinterpret_cast<bf4 *>(p.dv + out + 32 * db + 8 * g + 4 * half) = v;
    }
}

// Sum the terms of the blocks that have them, in their order: a thread for 4
// elements of a key, a workgroup for 1024 of the elements of a (batch row, key
// head) block of 32 keys.
template <int D>
__global__ void __launch_bounds__(256) swa_parts_kernel(const SwaParams p, const SwaBwdPlan plan) {
  const unsigned nkv = static_cast<unsigned>(p.nkv), per = plan.sum_blocks * 4;
  const int i = static_cast<int>(blockIdx.x % (D / 32)) * 256 + threadIdx.x;
  const unsigned id = blockIdx.x / (D / 32), bc = id / per, b32 = id % per, block = b32 / 4;
  const int64_t b = bc / nkv, c = bc % nkv;
  const int len = row_length(p, b), L = static_cast<int>(p.seqlen), j = static_cast<int>(b32) * 32 + i / (D / 4);
  if (j >= L) return;
  const float4 *main = reinterpret_cast<const float4 *>(
      p.ws_part + (static_cast<int64_t>(bc) * plan.sum_blocks + block) * plan.slices * 2 * 128 * D + (b32 % 4) * 32 * D) + i;
  const unsigned nfar = b32 < plan.far_blocks ? plan.far_chunks : 0;
  const float4 *far = reinterpret_cast<const float4 *>(
      p.ws_far + (static_cast<int64_t>(bc) * plan.far_blocks + b32) * plan.far_chunks * 2 * 32 * D) + i;
  float4 a = make_float4(0, 0, 0, 0), v = a;
  for (unsigned k = 0; k < plan.slices; ++k) {
    add(a, main[k * (2 * 128 * D / 4)]);
    add(v, main[k * (2 * 128 * D / 4) + 128 * D / 4]);
  }
#pragma unroll 4
  for (unsigned k = 0; k < nfar; ++k) {
    add(a, far[k * (2 * 32 * D / 4)]);
    add(v, far[k * (2 * 32 * D / 4) + 32 * D / 4]);
  }
  const float keep = j < len ? 1.0f : 0.0f, ka = keep * p.scale;
  const int64_t out = ((b * p.seqlen + j) * p.nkv + c) * D + i % (D / 4) * 4;
  const bf4 oa = {static_cast<__bf16>(a.x * ka), static_cast<__bf16>(a.y * ka), static_cast<__bf16>(a.z * ka),
                  static_cast<__bf16>(a.w * ka)};
  const bf4 ov = {static_cast<__bf16>(v.x * keep), static_cast<__bf16>(v.y * keep), static_cast<__bf16>(v.z * keep),
                  static_cast<__bf16>(v.w * keep)};
  *reinterpret_cast<bf4 *>(p.dk + out) = oa;
  *reinterpret_cast<bf4 *>(p.dv + out) = ov;
}

template <int D>
hipError_t launch_d(const SwaParams &p, const SwaBwdPlan &plan, hipStream_t s) {
  const int64_t group = p.nheads / p.nkv;
  const int hw = group % 4 == 0 ? 4 : group % 2 == 0 ? 2 : 1;
  const int64_t qspan = 32 * (4 / hw), qtiles = (p.seqlen + qspan - 1) / qspan;
  const int64_t n = qtiles * (group / hw) * p.nkv * p.batch, items = plan.items * p.batch * p.nkv;
  hipLaunchKernelGGL((swa_dq_kernel<D>), dim3(static_cast<uint32_t>(n)), dim3(256), 0, s, p, hw,
                     static_cast<unsigned>(qtiles), static_cast<unsigned>(n));
  hipLaunchKernelGGL((swa_dkv_kernel<D>), dim3(static_cast<uint32_t>(items)), dim3(256), 0, s, p, plan,
                     static_cast<unsigned>(items));
  if (plan.sum_blocks > 0)
    hipLaunchKernelGGL((swa_parts_kernel<D>), dim3(static_cast<uint32_t>(plan.sum_blocks * 4 * (D / 32) * p.batch * p.nkv)), dim3(256), 0, s,
                       p, plan);
  return hipGetLastError();
}

}  // namespace

SwaBwdPlan swa_bwd_plan(int64_t batch, int64_t seqlen, int64_t nheads, int64_t nkv, int64_t headdim, int64_t window,
                        int64_t sinks) {
  SwaBwdPlan plan{};
  const int64_t blocks = (seqlen + 127) / 128, group = nheads / nkv;
  window = window < seqlen ? window : seqlen;
  sinks = sinks < seqlen ? sinks : seqlen;
  plan.blocks = static_cast<unsigned>(blocks);
  // Too few workgroups for the 256 CUs, or for uneven ones to even out: the heads
  // of a group are shared out (8192 tokens, 16 heads of 128 on 4: window 1024
  // 311 us, with four times as many workgroups 351; window 8192 1547 and 1146).
  const int64_t want = (headdim == 64 ? 512 : 256) * (uneven(window, seqlen) ? 4 : 1);
  int64_t slices = 1;
  while (slices < group && batch * nkv * blocks * slices < want) {
    do ++slices;
    while (group % slices != 0);
  }
  plan.slices = static_cast<unsigned>(slices);
  // Far items, where queries lie past the first block's window: about six
  // (32 queries, head) pairs per wavefront.
  const int64_t pairs = ((seqlen + 31) / 32 - 2 * ((window + 127 + kTile - 1) / kTile)) * group;
  if (sinks > 0 && pairs > 0) {
    plan.far_blocks = static_cast<unsigned>((sinks + 31) / 32);
    // No more than 2048 workgroups in all, or one per block: every chunk has
    // terms of its own, which with thousands of sinks would grow as sinks x seqlen.
    const int64_t rows = batch > 0 ? batch * nkv : 1, most = 2048 / (rows * plan.far_blocks), chunks = (pairs + 23) / 24;
    plan.far_chunks = static_cast<unsigned>(chunks < most ? chunks : most > 1 ? most : 1);
  }
  const int64_t sink_blocks = plan.far_blocks > 0 ? (sinks + 127) / 128 : 0;
  plan.sum_blocks = static_cast<unsigned>(slices > 1 ? blocks : sink_blocks);
  plan.items = static_cast<int64_t>(plan.far_blocks) * plan.far_chunks + blocks * slices;
  return plan;
}

hipError_t launch_swa_bwd(const SwaParams &p, const SwaBwdPlan &plan, hipStream_t s) {
  return p.headdim == 64 ? launch_d<64>(p, plan, s) : launch_d<128>(p, plan, s);
}

}  // namespace ssmb
