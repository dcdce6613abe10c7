// Sliding-window attention with sinks for gfx950, forward.
//
// Query t sees key j when j <= t < length and (t - j < window or j < sinks):
//   y_t = sum_j exp(scale q_t.k_j) v_j / sum_j exp(scale q_t.k_j)
// in one pass over the keys with a running maximum and sum.
//
// A wavefront takes 32 queries of one head; the four of a workgroup share
// tiles of 64 keys and values in LDS and take up to four heads of a group
// over the same 32 queries (few tiles that only part of the workgroup sees)
// or up to 128 queries of one head.  S^T = K Q^T leaves a query's scores in
// one lane (and its other half), so the softmax needs one exchange per tile,
// and p goes into O^T = V^T P^T as it lies (see swa_tile.h), rounded to bfloat16,
// which the matrix cores take.  That makes the error of y 2.1e-3 of its norm,
// where rounding y alone gives 1.65e-3; a second part of p, left over, would give
// that, and take 20 to 30% more time (8192 tokens, 16 heads of 128, window 1024:
// 85 -> 107 us; 4 x 4096 tokens over all their past, 32 heads of 64: 399 -> 520).
//
// Bound by the wavefronts' alternation of matrix instructions (busy 40% of the
// time) and softmax (30%), which overlap across the two or three wavefronts of
// a SIMD only: 8192 tokens, 16 heads of 128 on 4, window 1024, 82 us a call (790
// TFLOP/s); over all the past 325 us (850 TFLOP/s).  64 queries per wavefront
// would halve the operand reads from LDS; they leave registers for one or two
// wavefronts per SIMD, and took 131 us against 91 with headdim 128, 387 against
// 383 with 64 (4 x 4096 tokens over all the past, 32 heads on 8).
#include "swa_tile.h"

namespace ssmb {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// What a workgroup knows of its work.
struct FwdWork {
  const uint16_t *k, *v;  // of the key head
  int q0, q1, wq0;        // first and last query of the workgroup, first of this wavefront
  KeyRow row;             // the keys its queries see
  int len, tiles;
  float c2;               // |scale| log2(e)
};

// One pass over the keys: o and sum (of this lane's half of the keys) of the
// lane's query t, with weights 2^(c2 s - top).  Returns whether a tile that
// some query sees in part held an infinity or NaN among its values: their
// products with weights of 0 would reach queries that do not see them.  SAFE
// keeps them out of the product and adds what they are worth by themselves.
template <int D, bool SAFE>
__device__ __forceinline__ bool attend(const SwaParams &p, const FwdWork &w, u4 (&lds)[2][2][kTile * D / 8],
                                       const bf8 (&q)[D / 16], f16v (&o)[D / 32], float &top, float &sum, int tid) {
  constexpr int CH = D / 8, NB = D / 32, NS = D / 16;
  const int lane = tid & 63, half = lane >> 5, t = w.wq0 + (lane & 31);
  const int window = static_cast<int>(p.window), sinks = static_cast<int>(p.sinks);
  const Lanes at = lanes_of<D>(lane);
  unsigned bad = 0;
  top = -INFINITY;
  sum = 0.0f;
#pragma unroll
  for (int db = 0; db < NB; ++db) o[db] = f16v{};
  auto start = [&](int i) {
    load_keys<D, 256>(lds[i & 1][0], w.k, p.k_token, w.row, i * kTile, w.len - 1, tid);
    load_keys<D, 256>(lds[i & 1][1], w.v, p.v_token, w.row, i * kTile, w.len - 1, tid);
  };
  start(0);
  for (int i = 0; i < w.tiles; ++i) {
    wait_tiles();
    __syncthreads();  // tile i has landed, and nobody reads the other buffer any more
    if (i + 1 < w.tiles) start(i + 1);
    const int v0 = i * kTile, j0 = w.row.key(v0), j1 = w.row.key(v0 + kTile - 1);
    const u4 *kt = lds[i & 1][0], *vt = lds[i & 1][1];
    if constexpr (!SAFE) {
      if (j1 > w.q0 || w.q1 - j0 >= window) {  // some of the workgroup's queries see part of it: each wavefront looks at a quarter
#pragma unroll
        for (int k = 0; k < kTile * CH / 256; ++k) {
          const u4 v = vt[k * 256 + tid];
          bad |= not_finite(v[0]) | not_finite(v[1]) | not_finite(v[2]) | not_finite(v[3]);
        }
      }
    }
    // Does this wavefront see any of the tile, or all of it?
    if (j0 > w.wq0 + 31 || (j1 <= w.wq0 - window && j0 >= sinks) || w.wq0 >= w.len) continue;
    const bool whole = j1 <= w.wq0 && w.wq0 + 31 - j0 < window;
    f16v s[2] = {};
#pragma unroll
    for (int ks = 0; ks < NS; ++ks)
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) s[blk] = mfma(row_operand<D>(kt, 32 * blk, ks, at), q[ks], s[blk]);
    reads_ahead<2 * NS>();
    Seen seen = seen_by(w.row, t, v0, half, window, sinks);
    if (!whole) {
#pragma unroll
      for (int blk = 0; blk < 2; ++blk)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[blk][r] = seen(32 * blk + d_row(r, 0)) ? s[blk][r] : -INFINITY;
    }
    to_weights(s, w.c2, o, top, sum);
    if constexpr (SAFE) {
      if (!whole) {
        asm volatile("" : "+v"(seen.ahead), "+v"(seen.own));  // 32 masks are not to be kept for this
        bf8 vis[4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
          for (int e = 0; e < 8; ++e) vis[ks][e] = static_cast<__bf16>(seen(32 * (ks / 2) + d_row(ks % 2 * 8 + e, 0)) ? 1.0f : 0.0f);
        add_not_finite<D, 4, false>(vt, 0, vis, o, at);
      }
    }
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const bf8 pk = as_operand(s[ks / 2], ks % 2);
#pragma unroll
      for (int db = 0; db < NB; ++db) {
        bf8 v = col_operand<D>(vt, 16 * ks, db, at);
        if constexpr (SAFE) {
          if (!whole) v = only_finite(v);
        }
        o[db] = mfma(v, pk, o[db]);
        if constexpr (SAFE) __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  return (bad & 0x80008000u) != 0;
}

template <int D>
__global__ void __launch_bounds__(256, D == 64 ? 3 : 2) swa_fwd_kernel(const SwaParams p, int hw, unsigned qtiles, unsigned n) {
  constexpr int CH = D / 8, NB = D / 32, NS = D / 16;
  __shared__ __align__(16) u4 lds[2][2][kTile * CH];  // buffer, K or V
  __shared__ int found;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const unsigned nheads = static_cast<unsigned>(p.nheads), nkv = static_cast<unsigned>(p.nkv);
  const unsigned group = nheads / nkv, hb = group / hw;
  // Work order: query tile fastest, then head block of a key head, batch row, key head.
  const unsigned batch = static_cast<unsigned>(p.batch), id = xcd_order(blockIdx.x, n, nkv * batch);
  const unsigned rest = id / qtiles, qt = uneven(p.window, p.seqlen) ? qtiles - 1 - id % qtiles : id % qtiles;
  const int64_t c = rest / (hb * batch), b = rest / hb % batch;
  const int64_t head = c * group + (rest % hb) * hw + wave % hw;
  const int qspan = 32 * (4 / hw), q0 = static_cast<int>(qt) * qspan;
  FwdWork w;
  w.len = row_length(p, b);
  w.q0 = q0;
  w.q1 = q0 + qspan - 1;
  w.wq0 = q0 + 32 * (wave / hw);
  w.c2 = fmaxf(fabsf(p.scale) * kLog2e, 0x1p-100f);
  const int t = w.wq0 + (lane & 31), L = static_cast<int>(p.seqlen);  // t: this lane's query

  f16v o[NB] = {};
  float top = -INFINITY, sum = 0.0f;
  if (q0 < w.len) {
    const int last = w.len - 1, qlast = q0 + qspan - 1 < last ? q0 + qspan - 1 : last;
    w.k = p.k + b * p.k_batch + c * D;
    w.v = p.v + b * p.v_batch + c * D;
    w.row = key_row(q0, static_cast<int>(p.window), static_cast<int>(p.sinks));
    w.tiles = (w.row.first + qlast - w.row.low) / kTile + 1;
    bf8 q[NS];
    const int row = t < last ? t : last;
    const u4 *src = reinterpret_cast<const u4 *>(p.q + b * p.q_batch + row * p.q_token + head * D);
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      u4 v = src[2 * s + half];
      if (p.scale < 0.0f) v ^= 0x80008000u;  // a negative scale is taken as -q
      q[s] = __builtin_bit_cast(bf8, v);
    }
    if (tid == 0) found = 0;  // before the first barrier in attend()
    const bool bad = attend<D, false>(p, w, lds, q, o, top, sum, tid);
    if (__any(bad)) found = 1;
    __syncthreads();
    if (found) attend<D, true>(p, w, lds, q, o, top, sum, tid);
  }
  sum += other_half(sum);
  if (t >= L) return;
  const bool none = t >= w.len || sum == 0.0f;
  const float inv = none ? 0.0f : 1.0f / sum;
  uint16_t *out = p.y + ((b * p.seqlen + t) * p.nheads + head) * D;
#pragma unroll
  for (int db = 0; db < NB; ++db)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf4 v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = static_cast<__bf16>(none ? 0.0f : o[db][4 * j + r] * inv);
      *reinterpret_cast<bf4 *>(out + 32 * db + 8 * j + 4 * half) = v;
    }
  if (p.lse != nullptr && half == 0)
    p.lse[(b * p.nheads + head) * p.seqlen + t] = none ? -INFINITY : top * kLn2 + logf(sum);
}

}  // namespace

hipError_t launch_swa_fwd(const SwaParams &p, hipStream_t s) {
  const int64_t group = p.nheads / p.nkv;
  const int hw = group % 4 == 0 ? 4 : group % 2 == 0 ? 2 : 1;
  const int64_t qspan = 32 * (4 / hw), qtiles = (p.seqlen + qspan - 1) / qspan;
  const int64_t n = qtiles * (group / hw) * p.nkv * p.batch;
  const dim3 g(static_cast<uint32_t>(n)), t(256);
  const unsigned qt = static_cast<unsigned>(qtiles), un = static_cast<unsigned>(n);
  if (p.headdim == 64) hipLaunchKernelGGL((swa_fwd_kernel<64>), g, t, 0, s, p, hw, qt, un);
  else hipLaunchKernelGGL((swa_fwd_kernel<128>), g, t, 0, s, p, hw, qt, un);
  return hipGetLastError();
}

}  // namespace ssmb
